// Products with MXFP4 weights, Y[m][n] = sum_k X[m][k] W[n][k].
//
//   X MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4, e2m1 x e2m1, both blocks'
//     powers of two applied by the instruction; fp32 accumulation.
//   X bf16: the codes become bf16 with their power of two
//     (v_cvt_scalef32_pk_bf16_fp4, exact: two significant bits) in
//     registers, v_mfma_f32_16x16x32_bf16; fp32 accumulation.
//
// Both operands of the 16x16x128 MFMA hold 32 consecutive k per lane, so the
// order of k inside a lane is free as long as A and B agree: lane r + 16 q,
// word j of its codes, is k = 128 g + 32 q + 8 j .. + 7, and the bf16 MFMA of
// word j takes X[m][128 g + 32 q + 8 j .. + 7] from lane m + 16 q.
#include <hip/hip_runtime.h>

#include "mx.hpp"

namespace lowbit {
namespace {

struct MxArgs {
  int64_t M, N, K, ld;       // ld: elements between bf16 X rows
  const uint8_t* wc;         // packed weight codes / exponents
  const uint8_t* ws;
  const uint8_t* x;          // bf16 rows, or packed MXFP4 codes
  const uint8_t* xs;         // packed MXFP4 exponents of X
  void* y;
  int64_t G, GQ, NB, MB;     // groups, quads, row-blocks of W and of X
};

template <int T>
__device__ __forceinline__ v4f mfma_mx(const mx_u4& a, const mx_u4& b, const v4f& c, uint32_t sa, uint32_t sb) {
  const v8i A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const v8i B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, T, (int)sa, T, (int)sb);
}

// the 8 codes of one word as bf16, times 2^(eb - 127) (eb 0 .. 255; 255 gives NaN)
__device__ __forceinline__ v8bf bf16x8(uint32_t w, float s) {
  union {
    v2bf h[4];
    v8bf v;
  } r;
  r.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
  r.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
  r.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
  r.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  return r.v;
}
__device__ __forceinline__ float scale_float(uint32_t word, int t) {
  return __uint_as_float(((word >> (8 * t)) & 255u) << 23);
}

template <int YK>
__device__ __forceinline__ void store_y(void* y, int64_t i, float v) {
  if constexpr (YK == YK_F32) ((float*)y)[i] = v;
  else ((uint16_t*)y)[i] = (uint16_t)bf16_bits(v);
}

// ---------------------------------------------------------- few rows of X
// One workgroup of up to 16 waves per (RB row-blocks of W, 16 MT rows of X);
// the waves split the quads of K, each issues a whole quad's loads at once,
// and the partial tiles are added over the waves in a fixed order.
constexpr int kSmallWaves = 12;

template <bool X4, int MT, int RB, int YK>
__global__ __launch_bounds__(64 * kSmallWaves) void mx_small(MxArgs a) {
  extern __shared__ __attribute__((aligned(16))) float red[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, W = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int64_t rb0 = (int64_t)blockIdx.x * RB, mb0 = (int64_t)blockIdx.y * MT;
  v4f acc[MT][RB];
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < RB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int64_t gq = wave; gq < a.GQ; gq += W) {
    mx_u4 wc[RB][4];
    uint32_t wsc[RB];
#pragma unroll
    for (int j = 0; j < RB; j++) {
      const int64_t rb = rb0 + j < a.NB ? rb0 + j : a.NB - 1;
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const int64_t g = 4 * gq + t;
        wc[j][t] = mx_u4{0, 0, 0, 0};
        if (g < a.G)
          wc[j][t] = __builtin_nontemporal_load((const mx_u4*)(a.wc + ((rb * a.G + g) * 64 + lane) * 16));
      }
      wsc[j] = *(const uint32_t*)(a.ws + ((rb * a.GQ + gq) * 64 + lane) * 4);
    }
    if constexpr (X4) {
#pragma unroll
      for (int i = 0; i < MT; i++) {
        const int64_t mb = mb0 + i < a.MB ? mb0 + i : a.MB - 1;
        const uint32_t xsc = *(const uint32_t*)(a.xs + ((mb * a.GQ + gq) * 64 + lane) * 4);
        mx_u4 xc[4];
#pragma unroll
        for (int t = 0; t < 4; t++) {
          const int64_t g = 4 * gq + t;
          xc[t] = mx_u4{0, 0, 0, 0};
          if (g < a.G) xc[t] = *(const mx_u4*)(a.x + ((mb * a.G + g) * 64 + lane) * 16);
        }
#pragma unroll
        for (int j = 0; j < RB; j++) {
          acc[i][j] = mfma_mx<0>(xc[0], wc[j][0], acc[i][j], xsc, wsc[j]);
          acc[i][j] = mfma_mx<1>(xc[1], wc[j][1], acc[i][j], xsc, wsc[j]);
          acc[i][j] = mfma_mx<2>(xc[2], wc[j][2], acc[i][j], xsc, wsc[j]);
          acc[i][j] = mfma_mx<3>(xc[3], wc[j][3], acc[i][j], xsc, wsc[j]);
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        const int64_t k = gq * 512 + 128 * t + 32 * q;
        mx_u4 xv[MT][4];
#pragma unroll
        for (int i = 0; i < MT; i++) {
          const int64_t m = (mb0 + i) * 16 + r;
#pragma unroll
          for (int h = 0; h < 4; h++) xv[i][h] = mx_u4{0, 0, 0, 0};
          // rows of the tile are independent: only the lanes of real rows load
          if (m < a.M && k < a.K) {
            const mx_u4* src = (const mx_u4*)(a.x + (m * a.ld + k) * 2);
#pragma unroll
            for (int h = 0; h < 4; h++) xv[i][h] = src[h];
          }
        }
#pragma unroll
        for (int j = 0; j < RB; j++) {
          const float s = scale_float(wsc[j], t);
#pragma unroll
          for (int h = 0; h < 4; h++) {
            const v8bf b = bf16x8(wc[j][t][h], s);
#pragma unroll
            for (int i = 0; i < MT; i++)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, xv[i][h]), b,
                                                                  acc[i][j], 0, 0, 0);
          }
        }
      }
    }
  }
  // partial tiles to LDS, then added over the waves in order
  constexpr int TILES = MT * RB;
#pragma unroll
  for (int i = 0; i < MT; i++)
#pragma unroll
    for (int j = 0; j < RB; j++) *(v4f*)(red + ((wave * TILES + i * RB + j) * 64 + lane) * 4) = acc[i][j];
  __syncthreads();
  for (int it = threadIdx.x; it < TILES * 64; it += blockDim.x) {
    v4f s = *(const v4f*)(red + it * 4);
    for (int w = 1; w < W; w++) {
      const v4f v = *(const v4f*)(red + (w * TILES * 64 + it) * 4);
#pragma unroll
      for (int e = 0; e < 4; e++) s[e] += v[e];
    }
    const int tile = it >> 6, l = it & 63;
    const int64_t n = (rb0 + tile % RB) * 16 + (l & 15);
    if (n < a.N) {
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int64_t m = (mb0 + tile / RB) * 16 + 4 * (l >> 4) + e;
        if (m < a.M) store_y<YK>(a.y, m * a.N + n, s[e]);
      }
    }
  }
}

int small_waves(int64_t GQ) {
  const int64_t rounds = cdiv(GQ, kSmallWaves);
  return (int)cdiv(GQ, rounds);
}

template <bool X4, int MT, int RB>
void launch_small(const MxArgs& a, int ykind, hipStream_t s) {
  const int W = small_waves(a.GQ);
  const dim3 grid((unsigned)cdiv(a.NB, RB), (unsigned)cdiv(cdiv(a.M, 16), MT));
  const size_t lds = (size_t)W * MT * RB * 1024;
  if (ykind == YK_F32)
    hipLaunchKernelGGL((mx_small<X4, MT, RB, YK_F32>), grid, dim3(64 * W), lds, s, a);
  else
    hipLaunchKernelGGL((mx_small<X4, MT, RB, YK_BF16>), grid, dim3(64 * W), lds, s, a);
}

}  // namespace

hipError_t launch_gemm_mxfp4(const MxGemmArgs& g, hipStream_t s) {
  MxArgs a;
  a.M = g.M;
  a.N = g.N;
  a.K = g.K;
  a.ld = g.ld;
  a.wc = (const uint8_t*)g.pcodes;
  a.ws = (const uint8_t*)g.pscales;
  a.x = (const uint8_t*)g.x;
  a.xs = (const uint8_t*)g.x_pscales;
  a.y = g.y;
  a.G = mx_groups(g.K);
  a.GQ = mx_quads(g.K);
  a.NB = cdiv(g.N, 16);
  a.MB = cdiv(g.M, 16);
  if (g.x4) launch_small<true, 1, 1>(a, g.ykind, s);
  else launch_small<false, 1, 1>(a, g.ykind, s);
  return hipGetLastError();
}

}  // namespace lowbit
