// Writing new keys and values into the paged 8-bit cache.
//
// A page and head hold their keys' codes c and one e with value c 2^e (their
// values likewise).  For the new tokens of a page, e(a) is the smallest e
// >= -127 with a <= 448 2^e, a their largest finite magnitude; with earlier
// tokens in the page the exponent never falls, e = max(e_old, e(a)), and
// where it rises the earlier codes are multiplied by 2^(e_old - e) and
// rounded again (exact unless a code falls below e4m3's normal range).
// code = x / 2^e rounded to nearest even; an infinity becomes +-448, a NaN
// the NaN code; at e = 120 codes end at 240 (top_code).  x / 2^e is exact in
// fp32, so codes and exponents do not depend on the order of anything.
//
// One workgroup per (sequence, page that receives tokens, head): it owns the
// page's codes and exponents of that head, keys and values.  The new elements
// are read once and stay in registers while their largest magnitude is found;
// V's codes change from token rows to dim rows through LDS.  3 x 4093 tokens, 8
// heads of 128: bf16 into pages of 16 20.2 us (75 MB: 3.7 TB/s; reading twice
// 26.0 us), of 64 19.1 (24.2), fp32 23.8 us (5.3 TB/s; 35.9); 4 heads of 256 into
// pages of 128 26.4 us (49.4).  Loads in a chain (length, page, elements) bound the
// small pages and one token a sequence (64 of them: 7.0 us).
#include <hip/hip_runtime.h>

#include "kv8.hpp"

namespace lowbit {
namespace {

__device__ __forceinline__ uint32_t finite_abs(uint32_t u) {
  u &= 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}
// exponent byte of e(a) for the bits of a (448 = 1.75 * 2^8)
__device__ __forceinline__ uint32_t page_byte(uint32_t a) {
  const int e = (int)(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e > 0 ? (uint32_t)e : 0u;
}
// The largest code of a page: 448, and where 448 2^e would lie beyond the finite
// numbers (byte 247, values of 1.75 2^127 and more) the one that stands for
// 1.875 2^127.  (Infinities in the cache would reach rows that do not see them, as 0
// times them.)
__device__ __forceinline__ float top_code(uint32_t byte) { return byte < 247u ? 448.0f : 240.0f; }
__device__ __forceinline__ float clamp_code(float v, float top) {
  return fabsf(v) > top ? copysignf(top, v) : v;  // NaN passes
}
// 2^-(byte - 127)
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// eight elements as they lie in memory
template <bool F32>
struct Raw8 {
  mx_u4 w[F32 ? 2 : 1];
  __device__ __forceinline__ void read(const uint8_t* p) {
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); i++) w[i] = *(const mx_u4*)(p + 16 * i);
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (F32) return __uint_as_float(w[e >> 2][e & 3]);
    return __uint_as_float(e & 1 ? w[0][e >> 1] & 0xFFFF0000u : w[0][e >> 1] << 16);
  }
};

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, (int)w, true);
}

// 2^-rise for codes written under an exponent `rise` lower; 0 from 127 on, where
// even 448 2^-rise rounds to no code (and 2^-rise leaves the exponent field)
__device__ __forceinline__ float rise_factor(uint32_t rise) {
  return rise < 127u ? __uint_as_float((127u - rise) << 23) : 0.f;
}

// four codes times f, rounded again
__device__ __forceinline__ uint32_t requantize4(uint32_t w, float f) {
  return codes4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * f, __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * f,
                __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * f, __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * f);
}

// HOLD: pieces of eight elements that a thread keeps between the search for the
// largest magnitude and the rounding; THREADS HOLD pieces are a page.
template <bool F32, int D, int THREADS, int HOLD>
__global__ __launch_bounds__(THREADS) void kv8_append(KvArgs a, int64_t span, const uint8_t* __restrict__ K,
                                                             const uint8_t* __restrict__ V, int64_t k_stride,
                                                             int64_t v_stride) {
  constexpr int E = F32 ? 4 : 2, D8 = D / 8;
  extern __shared__ __attribute__((aligned(16))) uint8_t vt[];  // [D][P + 4] codes of V: 2 lanes to a bank
  __shared__ uint32_t red[2][THREADS / 64];
  const int tid = threadIdx.x;
  const uint32_t H = (uint32_t)a.H, at = blockIdx.x / H, b = at / (uint32_t)span, j = at - b * (uint32_t)span;
  const int h = (int)(blockIdx.x - at * H);
  const int P = 1 << a.lp, VP = P + 4;
  const SeqSpan s = seq_span(a, b);
  const int first = s.len - s.n;  // negative: the earliest new tokens lie before the sequence
  const int lo0 = first > 0 ? first : 0;
  const int64_t slot = (lo0 >> a.lp) + j;
  const int base = (int)(slot << a.lp);
  const int lo = lo0 > base ? lo0 - base : 0;                     // new tokens of the page: [lo, hi)
  const int hi = s.len - base < P ? s.len - base : P;
  if (s.n == 0 || lo >= hi) return;
  const int64_t page = a.table[b * (int64_t)a.width + slot];
  if (page < 0 || page >= a.n_pages) {
    if (tid == 0 && a.bad) atomicAdd(a.bad, 1);
    return;
  }
  const int64_t row = s.row0 + (base - first);                    // row of the page's token 0
  const uint8_t* kp = K + (row * k_stride + (int64_t)h * D) * E;
  const uint8_t* vp = V + (row * v_stride + (int64_t)h * D) * E;

  const int pieces = (hi - lo) * D8;
  uint32_t ak = 0, av = 0;
  Raw8<F32> hk[HOLD], hv[HOLD];
#pragma unroll
  for (int c = 0; c < HOLD; c++) {
    const int i = tid + c * THREADS, t = lo + i / D8, d = (i % D8) * 8;
    if (i >= pieces) break;
    hk[c].read(kp + (t * k_stride + d) * E);
    hv[c].read(vp + (t * v_stride + d) * E);
  }
#pragma unroll
  for (int c = 0; c < HOLD; c++) {
    if (tid + c * THREADS >= pieces) break;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      ak = max(ak, finite_abs(__float_as_uint(hk[c][e])));
      av = max(av, finite_abs(__float_as_uint(hv[c][e])));
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
  for (int w = 0; w < THREADS / 64; w++) {
    ak = max(ak, red[0][w]);
    av = max(av, red[1][w]);
  }
  uint32_t bk = page_byte(ak), bv = page_byte(av);
  if (lo > 0) {
    bk = max(bk, ok);
    bv = max(bv, ov);
  }
  const float ik = inv_scale(bk), iv = inv_scale(bv), tk = top_code(bk), tv = top_code(bv);
  uint8_t* kc = a.kc + ph * P * D;
  uint8_t* vc = a.vc + ph * P * D;
#pragma unroll
  for (int c = 0; c < HOLD; c++) {
    const int i = tid + c * THREADS, t = lo + i / D8, d = (i % D8) * 8;
    if (i >= pieces) break;
    float x[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
      x[e] = clamp_code(hk[c][e] * ik, tk);
      y[e] = clamp_code(hv[c][e] * iv, tv);
    }
    *(uint2*)(kc + t * D + d) = make_uint2(codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7]));
    const uint32_t w0 = codes4(y[0], y[1], y[2], y[3]), w1 = codes4(y[4], y[5], y[6], y[7]);
#pragma unroll
    for (int e = 0; e < 4; e++) {
      vt[(d + e) * VP + t] = (uint8_t)(w0 >> (8 * e));
      vt[(d + 4 + e) * VP + t] = (uint8_t)(w1 >> (8 * e));
    }
  }
  // earlier tokens of the page, where its exponent rose
  if (lo > 0 && bk > ok) {
    const float f = rise_factor(bk - ok);
    for (int i = tid; i < lo * (D / 4); i += THREADS) {
      uint32_t* w = (uint32_t*)kc + i;
      *w = requantize4(*w, f);
    }
  }
  const bool rise = lo > 0 && bv > ov;
  const float fv = rise_factor(rise ? bv - ov : 0u);
  __syncthreads();
  // V rows of the page, four tokens at a time: whole words where all four are
  // written, else byte by byte (tokens behind the last one stay as they were)
  for (int i = tid; i < D * (P / 4); i += THREADS) {
    const int t = (i & (P / 4 - 1)) * 4;
    if (t >= hi || (t + 4 <= lo && !rise)) continue;
    uint32_t w = *(const uint32_t*)(vt + (i >> (a.lp - 2)) * VP + t);
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

// A page of one head in pieces of eight elements, a power of two from 128 to
// 4096: HOLD of them (1, 2 or 4) to a thread.
int64_t page_pieces(const KvArgs& a) { return ((int64_t)a.D << a.lp) / 8; }
int append_threads(int64_t pieces) { return pieces <= 1024 ? 256 : (int)(pieces / 4); }

template <bool F32, int D>
hipError_t launch_d(const KvArgs& a, int64_t span, const void* K, const void* V, int64_t ks, int64_t vs,
                    hipStream_t s) {
  const int64_t pieces = page_pieces(a);
  const dim3 grid((unsigned)(a.n_seqs * span * a.H)), block((unsigned)append_threads(pieces));
  const size_t lds = (size_t)D * ((1 << a.lp) + 4);
  const uint8_t *k = (const uint8_t*)K, *v = (const uint8_t*)V;
#define LOWBIT_APPEND(THREADS, HOLD) \
  hipLaunchKernelGGL((kv8_append<F32, D, THREADS, HOLD>), grid, block, lds, s, a, span, k, v, ks, vs)
  if (pieces <= 256) LOWBIT_APPEND(256, 1);
  else if (pieces <= 512) LOWBIT_APPEND(256, 2);
  else if (pieces <= 1024) LOWBIT_APPEND(256, 4);
  else if (pieces <= 2048) LOWBIT_APPEND(512, 4);
  else LOWBIT_APPEND(1024, 4);
#undef LOWBIT_APPEND
  return hipGetLastError();
}

}  // namespace

int64_t kv8_span(const KvArgs& a) { return ((a.max_q + (int64_t(1) << a.lp) - 2) >> a.lp) + 1; }

bool kv8_append_fits(const KvArgs& a) {
  const int64_t groups = a.n_seqs * kv8_span(a) * a.H;
  return groups <= (int64_t(1) << 23) && groups * append_threads(page_pieces(a)) <= kMaxThreads;
}

hipError_t launch_kv8_append(const KvArgs& a, bool f32, const void* K, const void* V, int64_t k_stride,
                             int64_t v_stride, hipStream_t s) {
  auto launch = [&](auto is32) {
    constexpr bool F32 = decltype(is32)::value;
    const int64_t span = kv8_span(a);
    return a.D == 64    ? launch_d<F32, 64>(a, span, K, V, k_stride, v_stride, s)
           : a.D == 128 ? launch_d<F32, 128>(a, span, K, V, k_stride, v_stride, s)
                        : launch_d<F32, 256>(a, span, K, V, k_stride, v_stride, s);
  };
  return f32 ? launch(std::true_type{}) : launch(std::false_type{});
}

}  // namespace lowbit
