// Norms of the heads of queries and keys, with the rotation by position.
//
// A head of D elements: y = x w / sqrt(mean x^2 + eps) (w NULL: y = x), then the
// pairs of the first 2 n_pairs elements, (i, i + n_pairs) or (2 i, 2 i + 1), turn
// by the angle position[axis(i)][token] freqs[i].  Squares, their sum and the
// turn are fp32; the angle is reduced to an eighth of a turn in fp64, so
// positions of any size keep their angle (fp32 would be off by 2^-24 of an angle
// of many turns), and its sine and cosine are Taylor series of an argument of at
// most pi / 4 (the first terms left out are below 2^-28 of the result).
//
// Bound by memory: 8191 x 28 heads of 256, fp32 to bf16, 76 us over two sets of inputs in
// turn (4.6 TB/s; a 4 GiB copy 4.7) and 74 over one, part of which the last-level cache
// keeps; 18432 x 40 heads of 128, bf16, three axes, adjacent pairs, 84.5 us (4.5 TB/s) and
// 79; one token, 48 heads of 128, 4.8 us (the launch, a load, the sums, a store).  Heads whose lanes are no
// power of two leave some idle: 16384 x 25 heads of 96 3.9 TB/s, of 72 3.2 TB/s (more
// loads on their way at once made those 5 to 25% slower).
//
// A wave has one token and a run of its heads.  Each lane finds the sine and
// cosine of one pair for all of the token's heads and leaves them in LDS.  A head
// lies in D / (2 W) lanes (rounded up to a power of two), two chunks of W
// elements each, so that a lane holds both elements of its pairs.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv8.hpp"

namespace lowbit {
namespace {

constexpr int kWaves = 4;       // of a workgroup
constexpr int kMaxPairs = 128;  // of a head (D <= 256)
constexpr int kHold = 4;        // heads of a lane read at once

// sin and cos of 2 pi s, |s| <= 1/8
__device__ __forceinline__ float2 small_turn(float s) {
  constexpr double t = 6.283185307179586;
  constexpr double t2 = t * t, t3 = t2 * t, t4 = t2 * t2, t5 = t4 * t, t6 = t3 * t3, t7 = t6 * t, t8 = t4 * t4;
  const float z = s * s;
  float p = fmaf(z, (float)(t8 * t / 362880), (float)(-t7 / 5040));
  p = fmaf(z, p, (float)(t5 / 120));
  p = fmaf(z, p, (float)(-t3 / 6));
  float q = fmaf(z, (float)(-t8 * t2 / 3628800), (float)(t8 / 40320));
  q = fmaf(z, q, (float)(-t6 / 720));
  q = fmaf(z, q, (float)(t4 / 24));
  q = fmaf(z, q, (float)(-t2 / 2));
  return make_float2(fmaf(s * z, p, s * (float)t), fmaf(z, q, 1.f));
}

// (cos, sin) of position f
__device__ __forceinline__ float2 turn_of(int position, double f) {
  double t = (double)position * f * 0.15915494309189535;  // turns
  t -= rint(t);
  const double e = rint(4. * t);
  const float2 v = small_turn((float)(t - 0.25 * e));  // sin, cos
  const int quarter = (int)e & 3;
  const float c = quarter & 1 ? v.x : v.y, s = quarter & 1 ? v.y : v.x;
  return make_float2(quarter == 1 || quarter == 2 ? -c : c, quarter >= 2 ? -s : s);
}

// W elements as they lie in memory
template <bool F32, int W>
struct Chunk {
  static constexpr int N = W * (F32 ? 4 : 2) / 8;  // words of 8 bytes
  uint2 w[N];
  __device__ __forceinline__ void read(const uint8_t* p) {
    if constexpr (N == 1) {
      w[0] = *(const uint2*)p;
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const mx_u4 v = *(const mx_u4*)(p + 8 * i);
        w[i] = make_uint2(v.x, v.y);
        w[i + 1] = make_uint2(v.z, v.w);
      }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (F32) return __uint_as_float(e & 1 ? w[e >> 1].y : w[e >> 1].x);
    const uint32_t u = e & 2 ? w[e >> 2].y : w[e >> 2].x;
    return __uint_as_float(e & 1 ? u & 0xFFFF0000u : u << 16);
  }
};
template <bool F32, int W>
__device__ __forceinline__ void write_chunk(uint8_t* p, const float* y) {
  uint32_t w[W * (F32 ? 4 : 2) / 4];
#pragma unroll
  for (int e = 0; e < W; e += F32 ? 1 : 2) {
    if constexpr (F32) {
      w[e] = __float_as_uint(y[e]);
    } else {
      v2bf h;
      h[0] = (__bf16)y[e];
      h[1] = (__bf16)y[e + 1];
      w[e / 2] = __builtin_bit_cast(uint32_t, h);
    }
  }
  constexpr int N = W * (F32 ? 4 : 2) / 4;
  if constexpr (N == 2) {
    *(uint2*)p = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(mx_u4*)(p + 4 * i) = mx_u4{w[i], w[i + 1], w[i + 2], w[i + 3]};
  }
}

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xF, 0xF, true));
}
// sum over the 2^lg neighbouring lanes of a head, the same in all of them
__device__ __forceinline__ float head_sum(float x, int lg) {
  if (lg >= 1) x = add_dpp<0xB1>(x);   // lane ^ 1
  if (lg >= 2) x = add_dpp<0x4E>(x);   // lane ^ 2
  if (lg >= 3) x = add_dpp<0x141>(x);  // the other four of eight
  if (lg >= 4) x = add_dpp<0x140>(x);  // the other eight of sixteen
  if (lg >= 5) x += __shfl_xor(x, 16);
  return x;
}

// 1 / sqrt(v), v >= 0, also where v is subnormal
__device__ __forceinline__ float inv_root(float v) {
  const bool small = v < 0x1p-100f;
  const float r = __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v);
  return small ? r * 0x1p32f : r;
}

// slices: parts of a token's heads, `per` of them each.  The wave's heads of all of
// its tokens are one row of passes (a pass: one head in each team), kHold of them
// on their way while one is worked on.
template <bool F32, bool OUT32, int W>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_rope(RopeArgs a, int lg, int slices, int per) {
  constexpr int EI = F32 ? 4 : 2, EO = OUT32 ? 4 : 2;
  __shared__ float2 turn_[kWaves][kMaxPairs];
  __shared__ __attribute__((aligned(16))) float weight_[2][2 * kMaxPairs];  // of queries and keys
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float2* turn = turn_[wave];
  const int team = lane >> lg, at = lane & ((1 << lg) - 1), teams = 64 >> lg;
  const bool mine = at * 2 * W < a.D;  // lanes behind the head's end idle
  // First dims of the lane's two chunks.  Pairs (i, i + n_pairs): one chunk has
  // their first elements, the other their second, where they turn; the dims behind
  // them lie in order.  Adjacent pairs: a chunk of either half of the head (both
  // chunks side by side: 4.3 TB/s in the place of 4.6).  Chunks turn or do not as a
  // whole: n_pairs is a multiple of W.
  const bool half = !a.adjacent && at * W < a.pairs;
  const int d0 = a.adjacent || half ? at * W : at * 2 * W;
  const int d1 = a.adjacent ? a.D / 2 + at * W : half ? a.pairs + at * W : d0 + W;
  const bool turn0 = half || (a.adjacent && d0 < 2 * a.pairs), turn1 = half || (a.adjacent && d1 < 2 * a.pairs);
  // the pair whose elements the lane has: e and W + e, or 2 e and 2 e + 1 of its 2 W
  auto pair_at = [&](int e) -> int { return !a.adjacent ? at * W + e : e < W / 2 ? d0 / 2 + e : d1 / 2 + e - W / 2; };
  const int heads = a.Hq + a.Hk, passes = (per + teams - 1) / teams;
  const int64_t items = a.tokens * slices, first = (int64_t)blockIdx.x * kWaves + wave, stride = (int64_t)gridDim.x * kWaves;

  struct Item {
    int64_t t;
    int h0, h_end;
  };
  auto item_at = [&](int64_t i) {
    Item x;
    x.t = slices > 1 ? i / slices : i;
    x.h0 = slices > 1 ? (int)(i - x.t * slices) * per : 0;
    x.h_end = min(heads, x.h0 + per);
    return x;
  };
  Chunk<F32, W> c0[kHold], c1[kHold];
  // what is read next: item and pass
  int64_t next = first;
  int next_pass = 0;
  Item ahead = item_at(next);
  auto read = [&](int slot) {
    if (next >= items) return;
    const int h = ahead.h0 + next_pass * teams + team;
    if (h < ahead.h_end && mine) {
      const uint8_t* p = h < a.Hq ? (const uint8_t*)a.q + (ahead.t * a.q_stride + h * a.D) * EI
                                  : (const uint8_t*)a.k + (ahead.t * a.k_stride + (h - a.Hq) * a.D) * EI;
      c0[slot].read(p + d0 * EI);
      c1[slot].read(p + d1 * EI);
    }
    if (++next_pass == passes) {
      next_pass = 0;
      next += stride;
      ahead = item_at(next);
    }
  };
#pragma unroll
  for (int e = 0; e < kHold; e++) {
    c0[e] = c1[e] = Chunk<F32, W>{};
    read(e);
  }
  // a lane's pairs are the same for every token
  constexpr int kMine = kMaxPairs / 64;
  double freq[kMine];
  int64_t row[kMine];  // of positions, -1: not rotated
  int pos[kMine];      // of the item to come
#pragma unroll
  for (int k = 0; k < kMine; k++) {
    const int i = lane + 64 * k;
    const int axis = i < a.pairs && a.pair_axis ? a.pair_axis[i] : 0;
    freq[k] = i < a.pairs ? a.freqs[i] : 0.;
    row[k] = i < a.pairs && axis >= 0 && axis < a.axes ? axis * a.pos_stride : -1;
  }
  // Bit e: its pair has no axis.  It is left out rather than turned by nothing: 0 times
  // an infinity would be NaN.
  uint32_t stay = 0;
  bool some_stay = false;
  if (a.pair_axis) {
#pragma unroll
    for (int e = 0; e < W; e++) {
      const int axis = mine && (e < W / 2 ? turn0 : turn1) ? a.pair_axis[pair_at(e)] : 0;
      stay |= axis >= 0 && axis < a.axes ? 0u : 1u << e;
    }
    some_stay = __any(stay != 0);
  }
  auto positions = [&](int64_t i) {
    const int64_t t = item_at(i).t;
#pragma unroll
    for (int k = 0; k < kMine; k++) pos[k] = row[k] >= 0 && i < items ? a.pos[row[k] + t] : 0;
  };
  positions(first);
  for (int d = threadIdx.x; d < a.D; d += 64 * kWaves) {
    weight_[0][d] = a.qw ? a.qw[d] : 1.f;
    weight_[1][d] = a.kw ? a.kw[d] : 1.f;
  }
  __syncthreads();

  float2 cs[W];
  int pass = 0;
  Item now;
  int64_t item = first;
  while (item < items) {
#pragma unroll
    for (int slot = 0; slot < kHold; slot++) {
      if (item >= items) break;
      if (pass == 0) {
        now = item_at(item);
#pragma unroll
        for (int k = 0; k < kMine; k++)
          if (64 * k < a.pairs) turn[lane + 64 * k] = turn_of(pos[k], freq[k]);
        positions(item + stride);
        // the wave's own LDS: its writes are done before its reads
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int e = 0; e < W; e++) {
          cs[e] = mine && (e < W / 2 ? turn0 : turn1) ? turn[pair_at(e)] : make_float2(1.f, 0.f);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      const int h = now.h0 + pass * teams + team;
      const bool is_q = h < a.Hq;
      float x[2 * W];
#pragma unroll
      for (int e = 0; e < W; e++) {
        x[e] = c0[slot][e];
        x[W + e] = c1[slot][e];
      }
      read(slot);
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * W; e++) sum = fmaf(x[e], x[e], sum);
      sum = head_sum(mine ? sum : 0.f, lg);
      if (h < now.h_end && mine) {
        if (is_q ? a.qw != nullptr : a.kw != nullptr) {
          const float r = inv_root(sum * a.inv_d + a.eps);
          const float* w = weight_[is_q ? 0 : 1];
#pragma unroll
          for (int e = 0; e < W; e += 4) {
            const v4f u = *(const v4f*)(w + d0 + e), v = *(const v4f*)(w + d1 + e);
#pragma unroll
            for (int f = 0; f < 4; f++) {
              x[e + f] = x[e + f] * r * u[f];
              x[W + e + f] = x[W + e + f] * r * v[f];
            }
          }
        }
        float y[2 * W];
#pragma unroll
        for (int e = 0; e < 2 * W; e++) y[e] = x[e];
        if (turn0) {
#pragma unroll
          for (int e = 0; e < W / 2; e++) {
            if (a.adjacent) {
              y[2 * e] = x[2 * e] * cs[e].x - x[2 * e + 1] * cs[e].y;
              y[2 * e + 1] = x[2 * e + 1] * cs[e].x + x[2 * e] * cs[e].y;
            } else {
              y[e] = x[e] * cs[e].x - x[W + e] * cs[e].y;
              y[W + e] = x[W + e] * cs[e].x + x[e] * cs[e].y;
            }
          }
        }
        if (turn1) {
#pragma unroll
          for (int e = W / 2; e < W; e++) {
            if (a.adjacent) {
              y[2 * e] = x[2 * e] * cs[e].x - x[2 * e + 1] * cs[e].y;
              y[2 * e + 1] = x[2 * e + 1] * cs[e].x + x[2 * e] * cs[e].y;
            } else {
              y[e] = x[e] * cs[e].x - x[W + e] * cs[e].y;
              y[W + e] = x[W + e] * cs[e].x + x[e] * cs[e].y;
            }
          }
        }
        if (some_stay) {
#pragma unroll
          for (int e = 0; e < W; e++) {
            const bool is = (stay >> e) & 1u;
            if (a.adjacent) {
              y[2 * e] = is ? x[2 * e] : y[2 * e];
              y[2 * e + 1] = is ? x[2 * e + 1] : y[2 * e + 1];
            } else {
              y[e] = is ? x[e] : y[e];
              y[W + e] = is ? x[W + e] : y[W + e];
            }
          }
        }
        uint8_t* p = is_q ? (uint8_t*)a.qo + (now.t * a.qo_stride + h * a.D) * EO
                          : (uint8_t*)a.ko + (now.t * a.ko_stride + (h - a.Hq) * a.D) * EO;
        write_chunk<OUT32, W>(p + d0 * EO, y);
        write_chunk<OUT32, W>(p + d1 * EO, y + W);
      }
      if (++pass == passes) {
        pass = 0;
        item += stride;
      }
    }
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& a, bool f32, bool out32, hipStream_t s) {
  const bool wide = a.D % 16 == 0 && a.pairs % 8 == 0;
  const int lanes = a.D / (wide ? 16 : 8);
  int lg = 0;
  while ((1 << lg) < lanes) lg++;
  const int teams = 64 >> lg, heads = a.Hq + a.Hk;
  // A wave takes all heads of a token where there are tokens for the whole chip,
  // else as few as are read at once, or one each.
  constexpr int64_t kFill = 8192;
  int per = heads;
  if (a.tokens < kFill) {
    const int64_t slices = std::min<int64_t>(cdiv(heads, teams), cdiv(kFill, a.tokens));
    per = (int)(cdiv(cdiv(heads, slices), teams) * teams);
  }
  const int slices = (int)cdiv(heads, per);
  // What the chip holds at once (three workgroups a compute unit; six with the
  // smaller chunks): a wave with several tokens reads ahead from one to the next.
  // 8191 x 28 heads of 256, fp32 to bf16, one set of inputs: 74 us, with a wave for each token 86.
  const int64_t blocks = std::min<int64_t>(cdiv(a.tokens * slices, kWaves), wide ? 768 : 1536);
  const dim3 grid((unsigned)blocks), block(64 * kWaves);
  auto go = [&](auto in, auto out) {
    constexpr bool I = decltype(in)::value, O = decltype(out)::value;
    if (wide) hipLaunchKernelGGL((qk_norm_rope<I, O, 8>), grid, block, 0, s, a, lg, slices, per);
    else hipLaunchKernelGGL((qk_norm_rope<I, O, 4>), grid, block, 0, s, a, lg, slices, per);
  };
  if (f32) out32 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  else out32 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace lowbit
