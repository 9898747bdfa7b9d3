// Writing new keys and values into the paged 8-bit cache.
//
// A page and head hold their keys' codes c and one e with value c 2^e (their
// values likewise).  For the new tokens of a page, e(a) is the smallest e
// >= -127 with a <= 448 2^e, a their largest finite magnitude; with earlier
// tokens in the page the exponent never falls, e = max(e_old, e(a)), and
// where it rises the earlier codes are multiplied by 2^(e_old - e) and
// rounded again (exact unless a code falls below e4m3's normal range).
// code = x / 2^e rounded to nearest even; an infinity becomes +-448, a NaN
// the NaN code.  x / 2^e is exact in fp32, so codes and exponents do not
// depend on the order of anything.
//
// One workgroup per (sequence, page that receives tokens, head): it owns the
// page's codes and exponents of that head, keys and values.
#include <hip/hip_runtime.h>

#include "kv8.hpp"

namespace lowbit {
namespace {

constexpr int kAppendThreads = 256;

__device__ __forceinline__ uint32_t finite_abs(uint32_t u) {
  u &= 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}
// exponent byte of e(a) for the bits of a (448 = 1.75 * 2^8)
__device__ __forceinline__ uint32_t page_byte(uint32_t a) {
  const int e = (int)(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}
__device__ __forceinline__ float clamp448(float v) {
  return fabsf(v) > 448.0f ? copysignf(448.0f, v) : v;  // NaN passes
}
// 2^-(byte - 127)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

template <bool F32>
__device__ __forceinline__ void read8(const uint8_t* p, float* v) {
  const mx_u4 a = *(const mx_u4*)p;
  if constexpr (F32) {
    const mx_u4 b = *(const mx_u4*)(p + 16);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, (int)w, true);
}

// four codes times 2^-shift, rounded again
__device__ __forceinline__ uint32_t requantize4(uint32_t w, float f) {
  return codes4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * f, __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * f,
                __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * f, __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * f);
}

template <bool F32, int D>
__global__ __launch_bounds__(kAppendThreads) void kv8_append(KvArgs a, int64_t span, const uint8_t* __restrict__ K,
                                                             const uint8_t* __restrict__ V, int64_t k_stride,
                                                             int64_t v_stride) {
  constexpr int E = F32 ? 4 : 2, D8 = D / 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];  // [D][P] codes of V
  __shared__ uint32_t red[2][kAppendThreads / 64];
  const int tid = threadIdx.x;
  const int64_t bid = blockIdx.x;
  const int h = (int)(bid % a.H);
  const int64_t j = (bid / a.H) % span, b = bid / a.H / span;
  const int P = 1 << a.lp;
  const SeqSpan s = seq_span(a, b);
  const int first = s.len - s.n;  // negative: the earliest new tokens lie before the sequence
  const int lo0 = first > 0 ? first : 0;
  const int64_t slot = (lo0 >> a.lp) + j;
  const int base = (int)(slot << a.lp);
  const int lo = lo0 > base ? lo0 - base : 0;                     // new tokens of the page: [lo, hi)
  const int hi = s.len - base < P ? s.len - base : P;
  if (s.n == 0 || lo >= hi) return;
  const int64_t page = a.table[b * a.width + slot];
  if (page < 0 || page >= a.n_pages) {
    if (tid == 0 && a.bad) atomicAdd(a.bad, 1);
    return;
  }
  const int64_t row = s.row0 + (base - first);                    // row of the page's token 0
  const uint8_t* kp = K + (row * k_stride + (int64_t)h * D) * E;
  const uint8_t* vp = V + (row * v_stride + (int64_t)h * D) * E;

  uint32_t ak = 0, av = 0;
  for (int i = tid; i < (hi - lo) * D8; i += kAppendThreads) {
    const int t = lo + i / D8, d = (i % D8) * 8;
    float x[8], y[8];
    read8<F32>(kp + (t * k_stride + d) * E, x);
    read8<F32>(vp + (t * v_stride + d) * E, y);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      ak = max(ak, finite_abs(__float_as_uint(x[e])));
      av = max(av, finite_abs(__float_as_uint(y[e])));
    }
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    ak = max(ak, (uint32_t)__shfl_xor((int)ak, m));
    av = max(av, (uint32_t)__shfl_xor((int)av, m));
  }
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = ak;
    red[1][tid >> 6] = av;
  }
  const int64_t ph = page * a.H + h;
  const uint32_t ok = a.ks[ph], ov = a.vs[ph];
  __syncthreads();  // also orders the exponents' reads before their writes below
#pragma unroll
  for (int w = 0; w < kAppendThreads / 64; w++) {
    ak = max(ak, red[0][w]);
    av = max(av, red[1][w]);
  }
  uint32_t bk = page_byte(ak), bv = page_byte(av);
  if (lo > 0) {
    bk = max(bk, ok);
    bv = max(bv, ov);
  }
  const float ik = inv_scale(bk), iv = inv_scale(bv);
  uint8_t* kc = a.kc + ph * P * D;
  uint8_t* vc = a.vc + ph * P * D;
  for (int i = tid; i < (hi - lo) * D8; i += kAppendThreads) {
    const int t = lo + i / D8, d = (i % D8) * 8;
    float x[8], y[8];
    read8<F32>(kp + (t * k_stride + d) * E, x);
    read8<F32>(vp + (t * v_stride + d) * E, y);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      x[e] = clamp448(x[e] * ik);
      y[e] = clamp448(y[e] * iv);
    }
    *(uint2*)(kc + t * D + d) = make_uint2(codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7]));
    const uint32_t w0 = codes4(y[0], y[1], y[2], y[3]), w1 = codes4(y[4], y[5], y[6], y[7]);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      vt[(d + e) * P + t] = (uint8_t)(w0 >> (8 * e));
      vt[(d + 4 + e) * P + t] = (uint8_t)(w1 >> (8 * e));
    }
  }
  // earlier tokens of the page, where its exponent rose
  if (lo > 0 && bk > ok) {
    const float f = inv_scale(bk - ok + 127);
    for (int i = tid; i < lo * (D / 4); i += kAppendThreads) {
      uint32_t* w = (uint32_t*)kc + i;
      *w = requantize4(*w, f);
    }
  }
  const bool rise = lo > 0 && bv > ov;
  const float fv = inv_scale(rise ? bv - ov + 127 : 127);
  __syncthreads();
  // V rows of the page, four tokens at a time: whole words where all four are
  // written, else byte by byte (tokens behind the last one stay as they were)
  for (int i = tid; i < D * (P / 4); i += kAppendThreads) {
    const int t = (i & (P / 4 - 1)) * 4;
    if (t >= hi || (t + 4 <= lo && !rise)) continue;
    uint32_t w = *(const uint32_t*)(vt + i * 4);
    if (t < lo && rise) {
      const uint32_t o = requantize4(*(const uint32_t*)(vc + i * 4), fv);
      const uint32_t keep = t + 4 <= lo ? 0xFFFFFFFFu : (1u << (8 * (lo - t))) - 1u;
      w = (o & keep) | (w & ~keep);
    }
    const int from = rise ? 0 : lo - t;  // first byte to write
    if (from <= 0 && t + 4 <= hi) {
      *(uint32_t*)(vc + i * 4) = w;
    } else {
      for (int e = from > 0 ? from : 0; e < 4 && t + e < hi; e++) vc[i * 4 + e] = (uint8_t)(w >> (8 * e));
    }
  }
  if (tid == 0) {
    a.ks[ph] = (uint8_t)bk;
    a.vs[ph] = (uint8_t)bv;
  }
}

template <bool F32>
hipError_t launch_d(const KvArgs& a, int64_t span, const void* K, const void* V, int64_t ks, int64_t vs,
                    hipStream_t s) {
  const dim3 grid((unsigned)(a.n_seqs * span * a.H));
  const size_t lds = (size_t)a.D << a.lp;
  const uint8_t *k = (const uint8_t*)K, *v = (const uint8_t*)V;
  if (a.D == 64) hipLaunchKernelGGL((kv8_append<F32, 64>), grid, dim3(kAppendThreads), lds, s, a, span, k, v, ks, vs);
  else if (a.D == 128) hipLaunchKernelGGL((kv8_append<F32, 128>), grid, dim3(kAppendThreads), lds, s, a, span, k, v, ks, vs);
  else hipLaunchKernelGGL((kv8_append<F32, 256>), grid, dim3(kAppendThreads), lds, s, a, span, k, v, ks, vs);
  return hipGetLastError();
}

}  // namespace

int64_t kv8_span(const KvArgs& a) { return ((a.max_q + (int64_t(1) << a.lp) - 2) >> a.lp) + 1; }

hipError_t launch_kv8_append(const KvArgs& a, bool f32, const void* K, const void* V, int64_t k_stride,
                             int64_t v_stride, hipStream_t s) {
  return f32 ? launch_d<true>(a, kv8_span(a), K, V, k_stride, v_stride, s)
             : launch_d<false>(a, kv8_span(a), K, V, k_stride, v_stride, s);
}

}  // namespace lowbit
