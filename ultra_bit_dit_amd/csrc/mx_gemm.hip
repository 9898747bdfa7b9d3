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

#include <algorithm>
#include <type_traits>

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
  int64_t MT, NT;            // tiles of X rows and of W rows
  uint32_t KS;               // splits of K
  float* part;               // partial tiles of the splits
  uint32_t* cnt;             // arrivals per tile
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
// Up to 16 bf16 or 32 MXFP4 rows: a workgroup per row-block of W and split of K,
// whose waves take the quads in turn.  A wave loads a quad's codes a quad ahead, straight to
// registers; bf16 rows of X reach the wave's own LDS as direct copies of 1 KiB
// (a row of a quad), with the 16-byte chunk c of row r at place c ^ r so that an
// operand's 16 rows fall on different banks.  The partial tiles are added over
// the waves in a fixed order.  1 x 5120 x 5120 5.5 us on the GPU (14 MB of
// codes), 5 x 5120 x 17408 15.2 us (47 MB, 3.1 TB/s: 320 workgroups on 256 compute
// units; with MXFP4 rows, so without widening the codes, 15.0), 1 x 34816 x 5120
// 21 us (4.5 TB/s).  32 MXFP4 rows x 5120 x 5120 8.7 us, x 15360 x 5120 14.3 us, x
// 700 x 17408 6.8 us (tiles: 12.7, 18.3 and 13.8); 17 bf16 rows here would need
// two operands' rows in every wave's LDS.
constexpr int kSmallWaves = 8;
constexpr int64_t kSmallRows = 16, kSmallRows4 = 32;  // bf16, MXFP4 X
constexpr int kSmallSplits = 8;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

__device__ __forceinline__ void copy16(const uint8_t* src, lds_u8* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

[[maybe_unused]] __device__ const mx_u4 mx_zeros[16] = {};

// RB: row-blocks of X (MXFP4 rows: up to two)
template <bool X4, int RB>
struct SmallQuad {
  mx_u4 w[4];
  uint32_t ws;
  mx_u4 x[RB][X4 ? 4 : 1];
  uint32_t xs[RB];
};

template <bool X4, int RB>
__device__ __forceinline__ void load_small(const MxArgs& a, int64_t rb, int64_t gq, int lane, SmallQuad<X4, RB>& o) {
  // groups past the last one read it again: their codes are cleared below
  const uint8_t* src = a.wc + rb * a.G * 1024 + 16 * lane;
#pragma unroll
  for (int t = 0; t < 4; t++)
    o.w[t] = __builtin_nontemporal_load((const mx_u4*)(src + min(4 * gq + t, a.G - 1) * 1024));
  o.ws = *(const uint32_t*)(a.ws + ((rb * a.GQ + gq) * 64 + lane) * 4);
  if constexpr (X4) {
#pragma unroll
    for (int i = 0; i < RB; i++) {
#pragma unroll
      for (int t = 0; t < 4; t++)
        o.x[i][t] = *(const mx_u4*)(a.x + ((i * a.G + min(4 * gq + t, a.G - 1)) * 64 + lane) * 16);
      o.xs[i] = *(const uint32_t*)(a.xs + ((i * a.GQ + gq) * 64 + lane) * 4);
    }
  }
}

// four floats, device-coherent
__device__ __forceinline__ void put_pairs(float* p, const v4f& v) {
#pragma unroll
  for (int e = 0; e < 2; e++)
    __hip_atomic_store((uint64_t*)p + e,
                       (uint64_t)__float_as_uint(v[2 * e]) | ((uint64_t)__float_as_uint(v[2 * e + 1]) << 32),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ v4f get_pairs(const float* p) {
  v4f v;
#pragma unroll
  for (int e = 0; e < 2; e++) {
    const uint64_t u = __hip_atomic_load((const uint64_t*)p + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v[2 * e] = __uint_as_float((uint32_t)u);
    v[2 * e + 1] = __uint_as_float((uint32_t)(u >> 32));
  }
  return v;
}

// lane l's four outputs of a 16 x 16 tile (rows m = 16 i + 4 (l / 16) .., column n = l % 16)
template <int YK>
__device__ __forceinline__ void store_small(const MxArgs& a, const v4f& s, int64_t rb, int i, int l) {
  const int64_t n = rb * 16 + (l & 15);
  if (n >= a.N) return;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const int64_t m = 16 * i + 4 * (l >> 4) + e;
    if (m < a.M) store_y<YK>(a.y, m * a.N + n, s[e]);
  }
}

template <bool X4, int RB, int YK>
__global__ __launch_bounds__(64 * kSmallWaves) void mx_small(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  extern __shared__ __attribute__((aligned(16))) uint8_t mem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  const int r = lane & 15, q = lane >> 4, rows = (int)a.M;
  const int64_t rb = blockIdx.x;
  const uint32_t ks = blockIdx.y, quads = (uint32_t)a.GQ;
  const int64_t q0 = quads * ks / a.KS, q1 = quads * (ks + 1) / a.KS;  // quads of this split
  uint8_t* xw = mem + wave * rows * 1024;
  v4f acc[RB][2] = {};  // two chains each
  const uint8_t* zeros = (const uint8_t*)mx_zeros;
  auto copy_x = [&](int64_t gq) {
    for (int m = 0; m < rows; m++) {
      const int64_t k = gq * 512 + 8 * (lane ^ m);
      copy16(k < a.K ? a.x + (m * a.ld + k) * 2 : zeros, (lds_u8*)xw + m * 1024);
    }
  };
  const int mrow = r < rows ? r : rows - 1;  // rows of the operand past the last one repeat it
  SmallQuad<X4, RB> cur, next;
  int64_t gq = q0 + wave;
  if (gq < q1) {
    if constexpr (!X4) copy_x(gq);
    load_small<X4, RB>(a, rb, gq, lane, cur);
  }
  for (; gq < q1; gq += W) {
    const bool more = gq + W < q1;
    // This quad's copies of X are the last loads issued: all are awaited here,
    // and the next quad's codes are loaded behind the first read.
    v8bf xf[2][4];
    auto read_x = [&](int t) {
#pragma unroll
      for (int h = 0; h < 4; h++)
        xf[t & 1][h] = *(const v8bf*)(xw + mrow * 1024 + (((16 * t + 4 * q + h) ^ mrow) * 16));
    };
    if constexpr (!X4) {
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      read_x(0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (more) load_small<X4, RB>(a, rb, gq + W, lane, next);
    if (4 * gq + 3 >= a.G) {
#pragma unroll
      for (int t = 1; t < 4; t++)
        if (4 * gq + t >= a.G) cur.w[t] = mx_u4{0, 0, 0, 0};
    }
    if constexpr (X4) {
#pragma unroll
      for (int i = 0; i < RB; i++) {
        acc[i][0] = mfma_mx<0>(cur.x[i][0], cur.w[0], acc[i][0], cur.xs[i], cur.ws);
        acc[i][1] = mfma_mx<1>(cur.x[i][1], cur.w[1], acc[i][1], cur.xs[i], cur.ws);
        acc[i][0] = mfma_mx<2>(cur.x[i][2], cur.w[2], acc[i][0], cur.xs[i], cur.ws);
        acc[i][1] = mfma_mx<3>(cur.x[i][3], cur.w[3], acc[i][1], cur.xs[i], cur.ws);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        if (t < 3) read_x(t + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 4; h++)
          acc[0][h & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              xf[t & 1][h], bf16x8(cur.w[t][h], scale_float(cur.ws, t)), acc[0][h & 1], 0, 0, 0);
      }
      if (more) {
        __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this quad's rows have been read
        copy_x(gq + W);
      }
    }
    if (more) cur = next;
  }
  // partial tiles to LDS, then added over the waves in order
  __syncthreads();
  float* red = (float*)mem;
#pragma unroll
  for (int i = 0; i < RB; i++) {
#pragma unroll
    for (int e = 0; e < 4; e++) acc[i][0][e] += acc[i][1][e];
    *(v4f*)(red + ((wave * RB + i) * 64 + lane) * 4) = acc[i][0];
  }
  __syncthreads();
  for (int i = wave; i < RB; i += W) {  // a wave for each row-block of X
    v4f s = *(const v4f*)(red + (i * 64 + lane) * 4);
    for (int w = 1; w < W; w++) {
      const v4f v = *(const v4f*)(red + ((w * RB + i) * 64 + lane) * 4);
#pragma unroll
      for (int e = 0; e < 4; e++) s[e] += v[e];
    }
    if (a.KS == 1) {
      store_small<YK>(a, s, rb, i, lane);
      continue;
    }
    // Splits of K: the last to arrive adds the partial tiles in their order.
    auto part = [&](int64_t k) -> float* { return a.part + (((k * a.NT + rb) * RB + i) * 64 + lane) * 4; };
    uint32_t* cnt = a.cnt + rb * RB + i;
    put_pairs(part(ks), s);
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
    uint32_t arrived = 0;
    if (lane == 0) arrived = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__builtin_amdgcn_readfirstlane((int)arrived) != (int)a.KS - 1) continue;
    if (lane == 0) __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v4f v[kSmallSplits];
#pragma unroll
    for (int k = 0; k < kSmallSplits; k++) v[k] = k < (int)a.KS ? get_pairs(part(k)) : v4f{0.f, 0.f, 0.f, 0.f};
    s = v[0];
#pragma unroll
    for (int k = 1; k < kSmallSplits; k++)
#pragma unroll
      for (int e = 0; e < 4; e++) s[e] += v[k][e];
    store_small<YK>(a, s, rb, i, lane);
  }
#endif
}

// Waves W of a workgroup and splits KS of K for NB row-blocks, GQ quads and M
// rows of X.  Four waves where the row-blocks alone fill the chip's 16 waves a
// compute unit, so that several workgroups share one and one starts while
// another ends (1 x 34816 x 5120: 21 us, 24 with 5 to 10 waves; 5 x 10240 x 5120:
// 9.6 us, 10.5 with eight), else eight (1 x 5120 x 5120: 5.5 us, 6.4 with four or
// ten; 5 x 2560 x 10240: 7.3 us with eight, 7.8 with seven that have equal turns,
// 9.8 with four), fewer where three workgroups' rows of X would not fit the LDS.
// K is split over workgroups where even so few waves run long: a join costs
// about 2.5 us, a wave's quad 1.25 (5 rows, 700 x 17408: 6.4 us, 8.5 without).
void plan_small(bool x4, int64_t M, int64_t NB, int64_t GQ, int* W_, int* KS_) {
  int64_t W = NB >= 640 ? 4 : 8;
  if (!x4) W = std::max<int64_t>(1, std::min(W, 48 / M));
  W = std::min(W, GQ);
  int64_t KS = 1;
  const int64_t turns = cdiv(GQ, W);
  if (turns >= 4 && NB * W < 1024) KS = std::min({(int64_t)kSmallSplits, turns, 4096 / (NB * W)});
  *W_ = (int)W;
  *KS_ = (int)KS;
}

template <bool X4, int RB>
void launch_small(const MxArgs& a, int W, int ykind, hipStream_t s) {
  const dim3 grid((unsigned)a.NT, (unsigned)a.KS);
  const size_t lds = (size_t)W * std::max<int64_t>(RB, X4 ? 0 : a.M) * 1024;
  if (ykind == YK_F32)
    hipLaunchKernelGGL((mx_small<X4, RB, YK_F32>), grid, dim3(64 * W), lds, s, a);
  else
    hipLaunchKernelGGL((mx_small<X4, RB, YK_BF16>), grid, dim3(64 * W), lds, s, a);
}

// ------------------------------------------------------------ many rows of X
// Workgroup tiles of 16 RN rows of W by 16 RM rows of X.  Codes, activations
// and exponents reach LDS as direct global -> LDS copies into a ring of group
// buffers; one counter of a wave's copies orders them, so each group waits
// exactly for its own (the later groups' stay in flight) and one barrier a
// group keeps the ring.  W is operand A (rows n) and X operand B (columns m):
// a lane then holds four consecutive n of one output row.
// s_waitcnt immediate: vmcnt n; lgkmcnt 0, so that a wave has what it read of a
// buffer before another refills it; expcnt at its maximum
constexpr int vm_wait(int n) { return (n & 15) | ((n >> 4) << 14) | 0x70; }

template <int N>
__device__ __forceinline__ void wait_copies_and_meet() {
  __asm__ volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vm_wait(N));
  __builtin_amdgcn_s_barrier();
  __asm__ volatile("" ::: "memory");
}

// Tile of workgroup bid: each XCD (bid % 8) takes a contiguous run of tiles,
// in bands of 8 row tiles of X with those running fastest, so that the
// workgroups of an XCD share both operands in its L2.
__device__ __forceinline__ void tile_of(uint32_t bid, uint32_t MT, uint32_t NT, int64_t* mt, int64_t* nt) {
  const uint32_t T = MT * NT, per = T / 8, rem = T % 8, x = bid % 8, i = bid / 8;
  const uint32_t t = x * per + (x < rem ? x : rem) + i;
  const uint32_t band = t / (8 * NT), left = MT - band * 8, w = left < 8 ? left : 8, r = t - band * 8 * NT;
  *mt = band * 8 + r % w;
  *nt = r / w;
}

// four consecutive outputs of row m from column n on
template <int YK>
__device__ __forceinline__ void store_quad(const MxArgs& a, int64_t m, int64_t n, const v4f& v) {
  if (a.N % 4 == 0 && n + 3 < a.N) {
    if constexpr (YK == YK_F32) {
      *(v4f*)((float*)a.y + m * a.N + n) = v;
    } else {
      uint2 w;
      w.x = bf16_bits(v[0]) | (bf16_bits(v[1]) << 16);
      w.y = bf16_bits(v[2]) | (bf16_bits(v[3]) << 16);
      *(uint2*)((uint16_t*)a.y + m * a.N + n) = w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (n + e < a.N) store_y<YK>(a.y, m * a.N + n + e, v[e]);
  }
}

// A wave's part of a tile: to Y, or with K split over workgroups to the
// workspace, [split][tile][part of a wave][thread], for mx_reduce to add.
template <int YK, int THREADS, int JN, int IM>
__device__ __forceinline__ void store_tile(const MxArgs& a, const v4f (&acc)[JN][IM], int64_t n0, int64_t m0, int64_t tile,
                                           uint32_t ks) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  if (a.KS > 1) {
    v4f* p = (v4f*)a.part + ((int64_t)ks * a.MT * a.NT + tile) * (JN * IM * THREADS) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < JN; j++)
#pragma unroll
      for (int i = 0; i < IM; i++) p[(j * IM + i) * THREADS] = acc[j][i];
    return;
  }
#pragma unroll
  for (int i = 0; i < IM; i++) {
    const int64_t m = m0 + 16 * i + r;
    if (m >= a.M) continue;
#pragma unroll
    for (int j = 0; j < JN; j++) store_quad<YK>(a, m, n0 + 16 * j + 4 * q, acc[j][i]);
  }
}

// The splits of K added in their order, four outputs a thread.  (The last
// split to arrive adding the others' tiles was slower: one workgroup reads
// KS tiles at 30 GB/s, 300 x 700 x 17408 in eight splits 12 us.)
template <int WN, int WM, int JN, int IM, int YK>
__global__ __launch_bounds__(256) void mx_reduce(MxArgs a) {
  constexpr int THREADS = 64 * WN * WM, PARTS = JN * IM;
  static_assert(THREADS % 256 == 0, "a block lies in one part of a tile");
  const uint32_t blk = blockIdx.x, per_tile = PARTS * THREADS / 256;
  const uint32_t tile = blk / per_tile, in = blk % per_tile, part = in / (THREADS / 256);
  const int tid = (in % (THREADS / 256)) * 256 + threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t mt, nt;
  tile_of(tile, (uint32_t)a.MT, (uint32_t)a.NT, &mt, &nt);
  const int wn = wave % WN, wm = wave / WN, j = part / IM, i = part % IM;
  const int64_t n = (nt * WN * JN + wn * JN + j) * 16 + 4 * (lane >> 4);
  const int64_t m = (mt * WM * IM + wm * IM + i) * 16 + (lane & 15);
  if (m >= a.M || n >= a.N) return;
  const int64_t step = a.MT * a.NT * (int64_t)(PARTS * THREADS);
  const v4f* p = (const v4f*)a.part + ((int64_t)tile * PARTS + part) * THREADS + tid;
  v4f s = p[0];
  for (uint32_t k = 1; k < a.KS; k++) {
    const v4f v = p[k * step];
#pragma unroll
    for (int e = 0; e < 4; e++) s[e] += v[e];
  }
  store_quad<YK>(a, m, n, s);
}

// X MXFP4.  WN x WM waves, each JN row-blocks of W by IM of X.  256 x 256 tiles:
// a group is 96 KiB of LDS reads and 1024 cycles of products on each SIMD, one after
// the other as all waves leave one barrier together; 128 x 128 where those would
// leave compute units idle.  4608 x 34816 x 5120 430 us (3.8 PFLOP/s) back to back:
// the MFMA is busy in 44% of the cycles, at 2.0 GHz.
template <int WN, int WM, int JN, int IM, int YK>
__global__ __launch_bounds__(64 * WN * WM) void mx_gemm4(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int RN = WN * JN, RM = WM * IM, R = RN + RM, WAVES = WN * WM, CP = R / WAVES;
  static_assert(R % WAVES == 0 && R / 4 == WAVES, "one scale copy and CP code copies per wave");
  // four group buffers; the first also holds the quad's exponents.  (Separate
  // objects, and no more of them: the compiler keeps apart the copies in flight
  // to four LDS objects and would wait for every copy before any read of a fifth.)
  __shared__ __attribute__((aligned(16))) uint8_t b0[R * 1280], b1[R * 1024], b2[R * 1024], b3[R * 1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN;
  int64_t mt, nt;
  const int64_t tile = blockIdx.x;
  const uint32_t ks = blockIdx.y, quads = (uint32_t)a.GQ;
  tile_of(blockIdx.x, (uint32_t)a.MT, (uint32_t)a.NT, &mt, &nt);
  // quads of this split; G: the end of its groups
  const int Q0 = (int)(quads * ks / a.KS), GQ = (int)(quads * (ks + 1) / a.KS);
  const int G0 = 4 * Q0, G = min(4 * GQ, (int)a.G);

  // this wave's code pieces: row-blocks CP wave .. of the tile's R (W first)
  const uint8_t* src[CP];
#pragma unroll
  for (int i = 0; i < CP; i++) {
    const int p = CP * wave + i;
    int64_t rb = p < RN ? nt * RN + p : mt * RM + (p - RN);
    const int64_t last = p < RN ? a.NB - 1 : a.MB - 1;
    rb = rb < last ? rb : last;
    src[i] = (p < RN ? a.wc : a.x) + rb * a.G * 1024 + 16 * lane;
  }
  // and four row-blocks' exponents
  const uint8_t* ssrc;
  {
    const int p = 4 * wave + (lane >> 4);
    int64_t rb = p < RN ? nt * RN + p : mt * RM + (p - RN);
    const int64_t last = p < RN ? a.NB - 1 : a.MB - 1;
    rb = rb < last ? rb : last;
    ssrc = (p < RN ? a.ws : a.xs) + rb * a.GQ * 256 + 16 * (lane & 15);
  }
  auto copy_group = [&](int g, uint8_t* buf) {
    const int64_t off = (int64_t)(g < G ? g : G - 1) * 1024;
#pragma unroll
    for (int i = 0; i < CP; i++) copy16(src[i] + off, (lds_u8*)buf + (CP * wave + i) * 1024);
    __builtin_amdgcn_sched_barrier(0);  // issued before the phase's products, not behind them
  };
  auto copy_scales = [&](int gq) {
    copy16(ssrc + (int64_t)(gq < GQ ? gq : GQ - 1) * 256, (lds_u8*)b0 + R * 1024 + wave * 1024);
  };

  v4f acc[JN][IM];
#pragma unroll
  for (int j = 0; j < JN; j++)
#pragma unroll
    for (int i = 0; i < IM; i++) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  uint32_t sw[JN], sx[IM];

  copy_scales(Q0);
  copy_group(G0, b0);
  __asm__ volatile("" ::: "memory");  // the waits below count the copies of each phase
  copy_group(G0 + 1, b1);
  __asm__ volatile("" ::: "memory");
  copy_group(G0 + 2, b2);

  auto compute = [&](auto tt, const uint8_t* buf) {
    constexpr int T = decltype(tt)::value;
    const uint8_t* pw = buf + wn * JN * 1024 + 16 * lane;
    const uint8_t* px = buf + (RN + wm * IM) * 1024 + 16 * lane;
    mx_u4 w[JN], x[IM];
#pragma unroll
    for (int j = 0; j < JN; j++) w[j] = *(const mx_u4*)(pw + j * 1024);
#pragma unroll
    for (int i = 0; i < IM; i++) x[i] = *(const mx_u4*)(px + i * 1024);
#pragma unroll
    for (int i = 0; i < IM; i++)
#pragma unroll
      for (int j = 0; j < JN; j++) acc[j][i] = mfma_mx<T>(w[j], x[i], acc[j][i], sw[j], sx[i]);
  };
  auto scales = [&]() {
    const uint8_t* buf = b0 + R * 1024 + 4 * lane;
#pragma unroll
    for (int j = 0; j < JN; j++) sw[j] = *(const uint32_t*)(buf + (wn * JN + j) * 256);
#pragma unroll
    for (int i = 0; i < IM; i++) sx[i] = *(const uint32_t*)(buf + (RN + wm * IM + i) * 256);
  };
  // Per quad, groups g .. g + 3 in buffers 0 .. 3.  Each phase waits until the
  // copies issued three phases ago are complete (the counts are those of the
  // two phases between), meets the other waves, which have then read the
  // previous buffer, and refills that one.  The next quad's exponents travel
  // with its first group, after every wave has read this quad's.
  auto phase0 = [&](int g) {
    wait_copies_and_meet<2 * CP>();
    copy_group(g + 3, b3);
    scales();
    compute(std::integral_constant<int, 0>{}, b0);
  };
  auto phase1 = [&](int g) {
    wait_copies_and_meet<2 * CP>();
    copy_group(g + 4, b0);
    copy_scales(g / 4 + 1);
    compute(std::integral_constant<int, 1>{}, b1);
  };
  auto phase2 = [&](int g) {
    wait_copies_and_meet<2 * CP + 1>();
    copy_group(g + 5, b1);
    compute(std::integral_constant<int, 2>{}, b2);
  };
  const int full = G & ~3;
  for (int g = G0; g < full; g += 4) {
    phase0(g);
    phase1(g);
    phase2(g);
    wait_copies_and_meet<2 * CP + 1>();
    copy_group(g + 6, b2);
    compute(std::integral_constant<int, 3>{}, b3);
  }
  if (full < G) phase0(full);
  if (full + 1 < G) phase1(full);
  if (full + 2 < G) phase2(full);
  // no copy may still be on its way to LDS when the workgroup ends
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  store_tile<YK, 64 * WAVES, JN, IM>(a, acc, (nt * RN + wn * JN) * 16, (mt * RM + wm * IM) * 16, tile, ks);
#endif
}

// X bf16.  WN x WM waves, each JN row-blocks of W by IM of X.  RING 2: two
// group buffers, the next group's copies in flight while one is multiplied
// (large tiles: 2048 cycles of MFMA per SIMD, longer than a copy takes).  RING
// 4: copies three groups ahead, for tiles that are multiplied faster than that.
// A row of X is 256 bytes of a group; its 16-byte chunk c lies at place
// c ^ (row % 16), so that the 16 rows of an operand read fall on different banks
// in pairs (places that keep all apart: the same time).  Chunks past K come
// from a block of zeros: the codes there are 0, but 0 times what follows a row
// of X need not be.  509 x 15360 x 5120 64 us (1.25 PFLOP/s, the rate of a large
// bf16 product), 4096 x 5120 x 5120 191 us.
template <int WN, int WM, int JN, int IM, int RING, int YK>
__global__ __launch_bounds__(64 * WN * WM) void mx_gemm16(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int RN = WN * JN, RM = WM * IM, WAVES = WN * WM;
  constexpr int CW = RN / WAVES, CX = 4 * RM / WAVES;  // code and X copies of a wave (1 KiB each)
  constexpr int CP = CW + CX;
  static_assert(CW * WAVES == RN && CX * WAVES == 4 * RM && RN / 4 <= WAVES, "whole copies per wave");
  static_assert(RING == 2 || RING == 4, "buffers of a quad's groups in turn");
  constexpr int XB = RM * 4096, CB = RN * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t b0[XB + CB + RN * 256], b1[XB + CB];
  __shared__ __attribute__((aligned(16))) uint8_t b2[RING == 4 ? XB + CB : 16], b3[RING == 4 ? XB + CB : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WN, wm = wave / WN, r = lane & 15, q = lane >> 4;
  int64_t mt, nt;
  const int64_t tile = blockIdx.x;
  const uint32_t ks = blockIdx.y, quads = (uint32_t)a.GQ;
  tile_of(blockIdx.x, (uint32_t)a.MT, (uint32_t)a.NT, &mt, &nt);
  // quads of this split; G: the end of its groups
  const int Q0 = (int)(quads * ks / a.KS), GQ = (int)(quads * (ks + 1) / a.KS);
  const int G0 = 4 * Q0, G = min(4 * GQ, (int)a.G);

  const uint8_t* wsrc[CW];
#pragma unroll
  for (int i = 0; i < CW; i++) {
    int64_t rb = nt * RN + CW * wave + i;
    rb = rb < a.NB - 1 ? rb : a.NB - 1;
    wsrc[i] = a.wc + rb * a.G * 1024 + 16 * lane;
  }
  // piece p of X: rows 4 p .. 4 p + 3; lane: row lane / 16, place lane % 16
  const uint8_t* xsrc[CX];
  int xk[CX];  // first k of the lane's chunk
#pragma unroll
  for (int i = 0; i < CX; i++) {
    const int row = 4 * (CX * wave + i) + (lane >> 4);
    int64_t m = mt * RM * 16 + row;
    m = m < a.M - 1 ? m : a.M - 1;
    xk[i] = 8 * ((lane & 15) ^ (row & 15));
    xsrc[i] = a.x + (m * a.ld + xk[i]) * 2;
  }
  // four row-blocks' exponents; waves past RN / 4 repeat another's copy, so
  // that all count the same copies
  const int sp = wave % (RN / 4);
  const uint8_t* ssrc;
  {
    int64_t rb = nt * RN + 4 * sp + (lane >> 4);
    rb = rb < a.NB - 1 ? rb : a.NB - 1;
    ssrc = a.ws + rb * a.GQ * 256 + 16 * (lane & 15);
  }
  const uint8_t* zeros = (const uint8_t*)mx_zeros;
  auto copy_group = [&](int g, uint8_t* buf) {
    g = g < G ? g : G - 1;
    const int left = (int)(a.K - (int64_t)g * 128 < 128 ? a.K - (int64_t)g * 128 : 128);
#pragma unroll
    for (int i = 0; i < CX; i++)
      copy16(xk[i] < left ? xsrc[i] + (int64_t)g * 256 : zeros, (lds_u8*)buf + (CX * wave + i) * 1024);
#pragma unroll
    for (int i = 0; i < CW; i++) copy16(wsrc[i] + (int64_t)g * 1024, (lds_u8*)buf + XB + (CW * wave + i) * 1024);
  };
  auto copy_scales = [&](int gq) {
    copy16(ssrc + (int64_t)(gq < GQ ? gq : GQ - 1) * 256, (lds_u8*)b0 + XB + CB + sp * 1024);
  };

  v4f acc[JN][IM];
#pragma unroll
  for (int j = 0; j < JN; j++)
#pragma unroll
    for (int i = 0; i < IM; i++) acc[j][i] = v4f{0.f, 0.f, 0.f, 0.f};
  uint32_t sw[JN];

  auto compute = [&](auto tt, const uint8_t* buf) {
    constexpr int T = decltype(tt)::value;
    const uint8_t* pw = buf + XB + wn * JN * 1024 + 16 * lane;
    const uint8_t* px = buf + wm * IM * 4096 + r * 256;
    mx_u4 w[JN];
    float s[JN];
#pragma unroll
    for (int j = 0; j < JN; j++) {
      w[j] = *(const mx_u4*)(pw + j * 1024);
      s[j] = scale_float(sw[j], T);
    }
#pragma unroll
    for (int h = 0; h < 4; h++) {
      v8bf x[IM], b[JN];
      const int at = ((4 * q + h) ^ r) * 16;
#pragma unroll
      for (int i = 0; i < IM; i++) x[i] = *(const v8bf*)(px + i * 4096 + at);
#pragma unroll
      for (int j = 0; j < JN; j++) b[j] = bf16x8(w[j][h], s[j]);
#pragma unroll
      for (int i = 0; i < IM; i++)
#pragma unroll
        for (int j = 0; j < JN; j++)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], x[i], acc[j][i], 0, 0, 0);
    }
  };
  auto scales = [&]() {
#pragma unroll
    for (int j = 0; j < JN; j++) sw[j] = *(const uint32_t*)(b0 + XB + CB + (wn * JN + j) * 256 + 4 * lane);
  };
  const int full = G & ~3;
  if constexpr (RING == 2) {
    // Each phase waits for its group (the only copies in flight), meets the
    // other waves, which have then read the other buffer, and refills that one.
    // The next quad's exponents travel behind every wave's read of this quad's.
    auto phase0 = [&](int g) {
      wait_copies_and_meet<0>();
      copy_group(g + 1, b1);
      __builtin_amdgcn_sched_barrier(0);
      scales();
      compute(std::integral_constant<int, 0>{}, b0);
    };
    auto phase1 = [&](int g) {
      wait_copies_and_meet<0>();
      copy_group(g + 2, b0);
      copy_scales(g / 4 + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 1>{}, b1);
    };
    auto phase2 = [&](int g) {
      wait_copies_and_meet<0>();
      copy_group(g + 3, b1);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 2>{}, b0);
    };
    copy_group(G0, b0);
    copy_scales(Q0);
    for (int g = G0; g < full; g += 4) {
      phase0(g);
      phase1(g);
      phase2(g);
      wait_copies_and_meet<0>();
      copy_group(g + 4, b0);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 3>{}, b1);
    }
    if (full < G) phase0(full);
    if (full + 1 < G) phase1(full);
    if (full + 2 < G) phase2(full);
  } else {
    // as mx_gemm4's phases: each waits for the copies issued three phases ago
    auto phase0 = [&](int g) {
      wait_copies_and_meet<2 * CP>();
      copy_group(g + 3, b3);
      __builtin_amdgcn_sched_barrier(0);
      scales();
      compute(std::integral_constant<int, 0>{}, b0);
    };
    auto phase1 = [&](int g) {
      wait_copies_and_meet<2 * CP>();
      copy_group(g + 4, b0);
      copy_scales(g / 4 + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 1>{}, b1);
    };
    auto phase2 = [&](int g) {
      wait_copies_and_meet<2 * CP + 1>();
      copy_group(g + 5, b1);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 2>{}, b2);
    };
    copy_scales(Q0);
    copy_group(G0, b0);
    __asm__ volatile("" ::: "memory");  // the waits count the copies of each phase
    copy_group(G0 + 1, b1);
    __asm__ volatile("" ::: "memory");
    copy_group(G0 + 2, b2);
    for (int g = G0; g < full; g += 4) {
      phase0(g);
      phase1(g);
      phase2(g);
      wait_copies_and_meet<2 * CP + 1>();
      copy_group(g + 6, b2);
      __builtin_amdgcn_sched_barrier(0);
      compute(std::integral_constant<int, 3>{}, b3);
    }
    if (full < G) phase0(full);
    if (full + 1 < G) phase1(full);
    if (full + 2 < G) phase2(full);
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  store_tile<YK, 64 * WAVES, JN, IM>(a, acc, (nt * RN + wn * JN) * 16, (mt * RM + wm * IM) * 16, tile, ks);
#endif
}

// Tile shapes, in row-blocks of X and of W.
struct Shape {
  int rm, rn;
};
constexpr Shape kBig4{16, 16}, kSmall4{8, 8}, kBig16{8, 16}, kSmall16{4, 8};

// What runs a product: few rows (small), or tiles of a shape with K in KS
// splits.
struct Plan {
  bool small;
  bool big;           // the larger tile
  bool resident;      // bf16, the smaller tile: two group buffers, three workgroups a compute unit
  int64_t MT, NT;     // small: NT row-blocks of W
  int KS, W;          // W: waves of a workgroup of few rows
  size_t part_bytes;
};

// MT 0: no choice fits a launch
Plan plan_gemm(bool x4, int64_t M, int64_t N, int64_t K) {
  Plan p{};
  if (M <= (x4 ? kSmallRows4 : kSmallRows)) {
    p.small = true;
    p.NT = cdiv(N, 16);
    plan_small(x4, M, p.NT, mx_quads(K), &p.W, &p.KS);
    p.part_bytes = p.KS > 1 ? (size_t)(p.NT * p.KS * cdiv(M, 16)) * 1024 : 0;
    return p;
  }
  const int64_t MB = cdiv(M, 16), NB = cdiv(N, 16), GQ = mx_quads(K);
  // Microseconds of each choice: rounds over the chip, a round the groups of a
  // split (`busy` where all compute units work, `idle` for few tiles; both
  // measured) and its start and end; a split adds a launch and the partial
  // tiles' way to memory and back.
  double best = 0;
  // The smaller bf16 tile also comes with two group buffers instead of four: a
  // group takes 0.7 us alone, but three workgroups share a compute unit at 0.5 us a
  // group each, so no round is left half empty (64 x 34816 x 5120: 41 us, 49 with
  // four buffers; 256 x 34816 x 5120: 100 and 121; 64 x 5120 x 17408: 32 and 26).
  for (int v = 0; v < (x4 ? 2 : 3); v++) {
    const bool big = v == 1, resident = v == 2;
    const Shape sh = x4 ? (big ? kBig4 : kSmall4) : (big ? kBig16 : kSmall16);
    const int64_t MT = cdiv(MB, sh.rm), NT = cdiv(NB, sh.rn), T = MT * NT;
    const int per_cu = x4 && !big ? 2 : 1;
    const double busy = x4 ? (big ? 1.0 : 0.6) : (big ? 1.53 : 0.51), idle = x4 ? (big ? 0.65 : 0.29) : (big ? 1.28 : 0.47);
    for (int KS = 1; KS <= 16; KS *= 2) {
      if (KS > 1 && (GQ < 2 * KS || T * KS > 1024)) break;
      if (T * (x4 && !big ? 256 : 512) > kMaxThreads) break;  // threads of its launch
      const double load = (double)(T * KS) / 256, groups = (double)cdiv(GQ, KS) * 4;
      const double split = KS > 1 ? 3.0 + (double)(T * KS) * sh.rm * sh.rn * 2048e-6 / 4.0 : 0.0;
      double c;
      if (resident) {
        const double group = 0.5 * (double)cdiv(T * KS, 256);
        c = groups * (group < 0.7 ? 0.7 : group) + 3.0 + split;
      } else {
        const double rounds = load <= per_cu ? 1.0 : (double)cdiv(T * KS, 256 * per_cu);
        const double group = load <= 1 ? idle + (busy - idle) * load * (per_cu == 1 ? 1.0 : 0.5) : busy;
        c = rounds * (groups * group + 2.5) + split;
      }
      if (best == 0 || c < best) {
        best = c;
        p.big = big;
        p.resident = resident;
        p.MT = MT;
        p.NT = NT;
        p.KS = KS;
        p.part_bytes = KS > 1 ? (size_t)(T * KS * sh.rm * sh.rn) * 1024 : 0;
      }
    }
  }
  return p;
}

template <int WN, int WM, int JN, int IM>
void launch_reduce(const MxArgs& a, int ykind, hipStream_t s) {
  const dim3 grid((unsigned)(a.MT * a.NT * JN * IM * WN * WM / 4));
  if (ykind == YK_F32) hipLaunchKernelGGL((mx_reduce<WN, WM, JN, IM, YK_F32>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((mx_reduce<WN, WM, JN, IM, YK_BF16>), grid, dim3(256), 0, s, a);
}

template <int WN, int WM, int JN, int IM>
void launch_tile4(const MxArgs& a, int ykind, hipStream_t s) {
  const dim3 grid((unsigned)(a.NT * a.MT), (unsigned)a.KS), block(64 * WN * WM);
  if (ykind == YK_F32) hipLaunchKernelGGL((mx_gemm4<WN, WM, JN, IM, YK_F32>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((mx_gemm4<WN, WM, JN, IM, YK_BF16>), grid, block, 0, s, a);
  if (a.KS > 1) launch_reduce<WN, WM, JN, IM>(a, ykind, s);
}
template <int WN, int WM, int JN, int IM, int RING>
void launch_tile16(const MxArgs& a, int ykind, hipStream_t s) {
  const dim3 grid((unsigned)(a.NT * a.MT), (unsigned)a.KS), block(64 * WN * WM);
  if (ykind == YK_F32) hipLaunchKernelGGL((mx_gemm16<WN, WM, JN, IM, RING, YK_F32>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((mx_gemm16<WN, WM, JN, IM, RING, YK_BF16>), grid, block, 0, s, a);
  if (a.KS > 1) launch_reduce<WN, WM, JN, IM>(a, ykind, s);
}

}  // namespace

bool gemm_mxfp4_fits(bool x4, int64_t M, int64_t N, int64_t K) {
  if (cdiv(M, 64) * cdiv(N, 128) < (int64_t(1) << 23)) return true;  // so many of the smallest tiles
  const Plan p = plan_gemm(x4, M, N, K);
  return p.small || p.MT > 0;
}

size_t gemm_mxfp4_workspace_bytes(bool x4, int64_t M, int64_t N, int64_t K) {
  const Plan p = plan_gemm(x4, M, N, K);
  return p.part_bytes ? (size_t)kCounterBytes + p.part_bytes : 0;
}

hipError_t launch_gemm_mxfp4(const MxGemmArgs& g, hipStream_t s) {
  const Plan p = plan_gemm(g.x4, g.M, g.N, g.K);
  MxArgs a{};
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
  a.MT = p.MT;
  a.NT = p.NT;
  a.KS = p.KS;
  if (p.part_bytes) {
    a.cnt = (uint32_t*)g.ws + 16;
    a.part = (float*)((uint8_t*)g.ws + kCounterBytes);
  }
  if (p.small) {
    if (!g.x4) launch_small<false, 1>(a, p.W, g.ykind, s);
    else if (g.M <= 16) launch_small<true, 1>(a, p.W, g.ykind, s);
    else launch_small<true, 2>(a, p.W, g.ykind, s);
  } else if (g.x4) {
    if (p.big) launch_tile4<4, 2, 4, 8>(a, g.ykind, s);
    else launch_tile4<2, 2, 4, 4>(a, g.ykind, s);
  } else {
    if (p.big) launch_tile16<4, 2, 4, 4, 2>(a, g.ykind, s);
    else if (p.resident) launch_tile16<4, 2, 2, 2, 2>(a, g.ykind, s);
    else launch_tile16<4, 2, 2, 2, 4>(a, g.ykind, s);
  }
  return hipGetLastError();
}

}  // namespace lowbit
