// MXFP4 (OCP microscaling: e2m1 codes, one E8M0 power of two per 32 values):
// quantizer and packer.
//
// Per block of 32 consecutive values of a row, a = max |x|:
//   e = max(floor(log2 a) - 2, -127), stored as the byte e + 127;
//   code = x / 2^e rounded to nearest even among 0, 0.5, 1, 1.5, 2, 3, 4, 6,
//   at most 6 in magnitude.
// x / 2^e is exact in fp32 (a power of two, and what underflows is far below
// the smallest midpoint 0.25), so the codes do not depend on any rounding
// but the last one.  A block holding an infinity or a NaN gets the byte 255
// (NaN) and codes 0.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "mx.hpp"

namespace lowbit {
namespace {

// The 8 elements at p (16 or 32 bytes) as floats.
template <bool F32>
struct Raw8 {
  mx_u4 a, b;
};
template <bool F32>
__device__ __forceinline__ void load8(const uint8_t* p, Raw8<F32>& r) {
  r.a = *(const mx_u4*)p;
  if constexpr (F32) r.b = *(const mx_u4*)(p + 16);
}
template <bool F32>
__device__ __forceinline__ void floats8(const Raw8<F32>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (F32) {
      v[i] = __uint_as_float(r.a[i]);
      v[4 + i] = __uint_as_float(r.b[i]);
    } else {
      v[2 * i] = __uint_as_float(r.a[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
    }
  }
}

// maximum over the four lanes 4 i .. 4 i + 3 (DPP quad permutations)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

// One wave quantizes one row-block over one quad (16 rows x 512 values).
// Load i of group t covers rows 4 i .. 4 i + 3, 256 contiguous bytes (bf16)
// of each: lane l holds the 8 values of piece l % 4 of block (l % 16) / 4 of
// row 4 i + l / 16, so a block's maximum is over four neighbouring lanes and
// the code words of one load are stored as four runs of 64 bytes.  Bound by
// memory: 5120 x 17408 bf16 with the values 83 us (404 MB, 4.85 TB/s, a copy's
// rate); one row of 5120 5.2 us, the way of one load and store.
template <bool F32>
__global__ __launch_bounds__(256) void quantize_mxfp4(int64_t rows, int64_t K, int64_t ld, int64_t units,
                                                      const uint8_t* __restrict__ X,
                                                      uint8_t* __restrict__ pcodes,
                                                      uint8_t* __restrict__ pscales,
                                                      uint8_t* __restrict__ values) {
  constexpr int E = F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t GQ = mx_quads(K), G = mx_groups(K);
  const int64_t rb = unit / GQ, gq = unit % GQ;
  const int q = (lane & 15) >> 2, p = lane & 3, rl = lane >> 4;
  const int64_t k0 = gq * 512 + 32 * q + 8 * p;

  Raw8<F32> raw[4][4];
#pragma unroll
  for (int t = 0; t < 4; t++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t row = rb * 16 + 4 * i + rl, k = k0 + 128 * t;
      raw[t][i].a = raw[t][i].b = mx_u4{0, 0, 0, 0};
      if (row < rows && k < K) load8<F32>(X + (row * ld + k) * E, raw[t][i]);
    }
  uint32_t ebytes[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int t = 0; t < 4; t++) {
    if (gq * 4 + t < G) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int64_t row = rb * 16 + 4 * i + rl, k = k0 + 128 * t;
        const bool in = row < rows && k < K;
        float v[8];
        floats8<F32>(raw[t][i], v);
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; j++) a = max(a, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        a = quad_max(a);
        // exponent byte of the maximum less 2, at least 0 (2^-127)
        const uint32_t ex = a >> 23;
        const bool bad = ex == 255u;
        const uint32_t eb = !in ? kMxUnitScale : bad ? 255u : ex > 2u ? ex - 2u : 0u;
        // 2^-e from its bits: the byte of -e is 254 - eb (in 2 .. 254)
        const float inv = __uint_as_float((254u - (bad ? 127u : eb)) << 23);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
        if (bad) w = 0;
        ebytes[i] |= eb << (8 * t);
        *(uint32_t*)(pcodes + ((rb * G + gq * 4 + t) * 64 + 4 * i + rl + 16 * q) * 16 + 4 * p) = w;
        if (values != nullptr && in) {
          uint8_t* o = values + (row * K + k) * E;
          const float s = bad ? __uint_as_float(0x7FC00000u)
                              : __uint_as_float(eb ? eb << 23 : 0x00400000u);
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; j++) {
            const uint32_t m = (w >> (4 * j)) & 7u;
            // e2m1 magnitude 0, .5, 1, 1.5, 2, 3, 4, 6 in half steps, four bits each
            const float mag = 0.5f * (float)((0xC8643210u >> (4 * m)) & 15u);
            f[j] = ((w >> (4 * j)) & 8u ? -mag : mag) * s;
          }
          mx_u4 b0, b1;
#pragma unroll
          for (int j = 0; j < 4; j++) {
            if constexpr (F32) {
              b0[j] = __float_as_uint(f[j]);
              b1[j] = __float_as_uint(f[4 + j]);
            } else {
              // exact: a code has two significant bits
              b0[j] = (__float_as_uint(f[2 * j]) >> 16) | (__float_as_uint(f[2 * j + 1]) & 0xFFFF0000u);
            }
          }
          *(mx_u4*)o = b0;
          if constexpr (F32) *(mx_u4*)(o + 16) = b1;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) ebytes[i] |= kMxUnitScale << (8 * t);
    }
  }
  // the four lanes of a block agree on its byte: lane p writes the word of load p
  const uint32_t word = p == 0 ? ebytes[0] : p == 1 ? ebytes[1] : p == 2 ? ebytes[2] : ebytes[3];
  *(uint32_t*)(pscales + ((rb * GQ + gq) * 64 + 4 * p + rl + 16 * q) * 4) = word;
}

// Row-major codes [rows][K/2] and exponent bytes [rows][K/32] into the tiled
// layout: one thread per (row, quad, block of the group), 4 blocks.
__global__ __launch_bounds__(256) void pack_mxfp4(int64_t rows, int64_t K, int64_t words,
                                                  const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales,
                                                  uint8_t* __restrict__ pcodes,
                                                  uint8_t* __restrict__ pscales) {
  const int64_t GQ = mx_quads(K), G = mx_groups(K);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int lane = (int)(i & 63);
    const int64_t u = i >> 6, rb = u / GQ, gq = u % GQ;
    const int64_t row = rb * 16 + (lane & 15);
    uint32_t eb = 0;
    for (int t = 0; t < 4; t++) {
      const int64_t g = gq * 4 + t, blk = 4 * g + (lane >> 4);
      const bool in = row < rows && blk * 32 < K;
      eb |= (in ? (uint32_t)scales[row * (K / 32) + blk] : kMxUnitScale) << (8 * t);
      if (g < G) {
        mx_u4 c{0, 0, 0, 0};
        if (in) c = *(const mx_u4*)(codes + row * (K / 2) + blk * 16);
        *(mx_u4*)(pcodes + ((rb * G + g) * 64 + lane) * 16) = c;
      }
    }
    *(uint32_t*)(pscales + i * 4) = eb;
  }
}

}  // namespace

namespace {
int64_t quantize_units(int64_t rows, int64_t K) { return cdiv(rows, 16) * mx_quads(K); }
}  // namespace

bool quantize_mxfp4_fits(int64_t rows, int64_t K) { return cdiv(quantize_units(rows, K), 4) * 256 <= kMaxThreads; }

hipError_t launch_quantize_mxfp4(int64_t rows, int64_t K, bool f32, const void* X, int64_t ld,
                                 void* pcodes, void* pscales, void* values, hipStream_t s) {
  const int64_t units = quantize_units(rows, K);
  const dim3 grid((unsigned)cdiv(units, 4));
  if (f32)
    hipLaunchKernelGGL(quantize_mxfp4<true>, grid, dim3(256), 0, s, rows, K, ld, units, (const uint8_t*)X,
                       (uint8_t*)pcodes, (uint8_t*)pscales, (uint8_t*)values);
  else
    hipLaunchKernelGGL(quantize_mxfp4<false>, grid, dim3(256), 0, s, rows, K, ld, units, (const uint8_t*)X,
                       (uint8_t*)pcodes, (uint8_t*)pscales, (uint8_t*)values);
  return hipGetLastError();
}

hipError_t launch_pack_mxfp4(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales,
                             void* pcodes, void* pscales, hipStream_t s) {
  const int64_t words = cdiv(rows, 16) * mx_quads(K) * 64;
  const int64_t blocks = std::min<int64_t>(cdiv(words, 256), 16384);
  hipLaunchKernelGGL(pack_mxfp4, dim3((unsigned)blocks), dim3(256), 0, s, rows, K, words, codes, scales,
                     (uint8_t*)pcodes, (uint8_t*)pscales);
  return hipGetLastError();
}

}  // namespace lowbit
