// MXFP4 operands (e2m1 codes, one power of two per block of 32), shared by
// the quantizer and the products (internal, not part of the public ABI).
//
// A row-block is 16 rows, a group 128 values of k, lane L = r + 16 q of a
// wavefront owns row r and block q of each group: its 32 codes are 16
// contiguous bytes and one operand of v_mfma_scale_f32_16x16x128_f8f6f4,
// and a group's 64 lanes are 1 KiB.  The exponent bytes of four groups (a
// quad) are one 32-bit word per lane, read by the MFMA's byte select.
#pragma once

#include "common.hpp"

namespace lowbit {

typedef unsigned int mx_u4 __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;
constexpr uint32_t kMxUnitScale = 127;  // 2^0: the exponent byte of padding

__host__ __device__ inline int64_t mx_groups(int64_t K) { return (K + 127) / 128; }
__host__ __device__ inline int64_t mx_quads(int64_t K) { return (K + 511) / 512; }

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// fp32 -> bf16 bits, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

}  // namespace lowbit
