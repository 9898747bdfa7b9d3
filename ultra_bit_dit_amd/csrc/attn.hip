// Attention over the paged 8-bit cache: O = softmax(scale Q K^T) V with
// K = 2^ek codes, V = 2^ev codes, per page and head.
//
// Rows.  The queries of one sequence that share a key / value head are one
// matrix of R = n G rows (n new tokens, G = query heads per key head): row
// rho is token rho / G, head h G + rho % G.
//
// Products run as v_mfma_f32_16x16x32_bf16 on codes widened to bf16 (exact,
// v_cvt_scalef32_pk_bf16_fp8), fp32 accumulation.  S^T = K Q^T puts a query
// row in lane n = L % 16 and tokens in the lane's registers; with the tile's
// token of row 4 g + j of tile t chosen as 16 g + 4 t + j, lane group
// g = L / 16 holds 16 consecutive tokens, which is what the B operand of
// O^T = V^T P^T needs: no exchange between the products, 16 tokens of one
// row of V are one 16-byte load, and (pages hold 16 tokens or more) one
// exponent ek and ev per lane and step.  Statistics, sums and O stay in fp32.
// Weights become bf16 for the second product: with few rows, where memory is the
// bound, in two terms, what the first leaves being the second (off by 2^-16 at
// most; 0.2 to 0.4 us a call more than one term, 1% of long ones, 5% with 32 rows a
// wave: 16 x 5 tokens in 2048, D = 64, 19.2 -> 20.1 us); with many rows, where the
// products are, rounded once (off by 2^-8 at most, the output's own rounding): a
// second term would take 2 x 4096 rows, 40 heads over 8, D = 128, from 383 to 497 us
// and attn_prompt32<64> out of its registers (221 -> 511 us).  Behind prefixes few rows
// of many sequences fill prompt tiles too: where a sequence has at most kFineRows of a
// key head, those have two terms as well (FINE; the batch of 64 below 90 -> 108 us, 45 x
// 5 tokens 42 -> 45, 16 with D = 256 101 -> 109).
//
// MODE.  kPlain: a call's rows see the tokens of one sequence each.  The others are
// of calls behind prefixes that groups of sequences share:
//   kBehind  a row's tokens are its prefix's and then its own, from two tables: steps
//            of the prefix come first, and the last one may be partly filled.  For
//            sequences of many rows, which fill tiles by themselves, and for small calls.
//   kHead    groups in the place of sequences: the rows of a group's sequences, which lie
//            in order, see its prefix, and leave their sums in the workspace;
//   kTail    each sequence's rows see its own tokens, and take those sums in.
// 64 single tokens behind 32760, 40 heads over 8, D = 128: 107 to 121 us by card and clock (kHead 97, 43 GFLOP
// and half as many again for the second terms, in tiles that five heads fill to 0.83; kTail 21, its chain of length,
// page, codes, sums); 16 behind two prefixes of 65000, 24 heads over 4, D = 256: 109 (86 + 29 alone); 45 x 5 tokens
// behind six of 8000, D = 64: 45 (25 + 21); 8 prompts of 777 behind 6001, 32 heads over 8, D = 128, in one kBehind
// launch and its join: 476 to 515 by card and clock (0.86 to 0.93 PFLOP/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "kv8.hpp"

namespace lowbit {
namespace {

enum Mode { kPlain, kBehind, kHead, kTail };

constexpr int kUnit = 64;  // tokens of one step of a wave
constexpr float kLn2 = 0.6931471805599453f;
// Results that are still to be joined lie in rows of kPartPad floats more than D:
// sums of O (before the division), maximum (of base 2), sum of weights.
constexpr int kPartPad = 4;

// eight codes times the power of two s as bf16 (exact: four significant bits)
__device__ __forceinline__ v8bf bf16x8_of_e4m3(uint32_t w0, uint32_t w1, float s) {
  union {
    v2bf h[4];
    v8bf v;
  } r;
  r.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
  r.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
  r.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
  r.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
  return r.v;
}
__device__ __forceinline__ float pow2_byte(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);  // byte 255: infinity, which no append writes
}
__device__ __forceinline__ v4f mfma(const v8bf& a, const v8bf& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// maximum over the four lanes of a row (n, n + 16, n + 32, n + 48): the swaps
// leave one of each pair in either result
__device__ __forceinline__ float group_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// eight bf16 numbers times 0: infinities and NaN become NaN
__device__ __forceinline__ mx_u4 zero_or_nan(mx_u4 w) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t lo = (w[i] & 0x7F80u) == 0x7F80u ? 0x7FC0u : 0u;
    const uint32_t hi = (w[i] & 0x7F800000u) == 0x7F800000u ? 0x7FC00000u : 0u;
    w[i] = (w[i] & 0x80008000u) | lo | hi;
  }
  return w;
}
// bytes of w that are e4m3 NaN codes (0x7F or 0xFF): bit 7 of each
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
// mask of the bytes of a word whose index e in 0..3 has lo <= e < hi
__device__ __forceinline__ uint32_t byte_range(int lo, int hi) {
  lo = lo < 0 ? 0 : lo > 4 ? 4 : lo;
  hi = hi < 0 ? 0 : hi > 4 ? 4 : hi;
  if (hi <= lo) return 0u;
  const uint32_t up = hi == 4 ? 0xFFFFFFFFu : (1u << (8 * hi)) - 1u;
  return up & ~((1u << (8 * lo)) - 1u);  // lo < 4 here
}

// a / b, a >= 0, b > 0: numbers are small but for the longest batches, and a
// 64-bit division takes some 150 instructions
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (__builtin_expect((((uint64_t)a | (uint64_t)b) >> 32) == 0, 1)) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// Up to 16 groups, one a lane, read before the sequences are known.
struct FirstGroups {
  int first = 0, last = 0, len = 0;
  __device__ __forceinline__ void read(const KvArgs& groups) {
    const int64_t i = threadIdx.x & 63;
    if (groups.n_seqs > 16 || i >= groups.n_seqs) return;
    first = groups.members ? groups.members[i] : (int)(i * groups.member_count);
    last = groups.members ? groups.members[i + 1] : (int)((i + 1) * groups.member_count);
    len = groups.lens[i];
  }
};

// The tokens of a sequence's shared prefix (kBehind; else none).  Positions count
// them first, in whole steps: own token t stands at kUnit * steps + t.
template <int MODE>
struct Head {
  int len = 0, steps = 0;
  const int32_t* table = nullptr;
  int64_t group = -1;
  __device__ __forceinline__ void take(const AttnArgs& a, int64_t g, int64_t n) {
    group = g;
    len = g < 0 ? 0 : (int)(n < 0 ? 0 : n < a.prefix.max_kv ? n : a.prefix.max_kv);
    steps = (len + kUnit - 1) / kUnit;
    table = a.prefix.table + (g < 0 ? 0 : g) * a.prefix.width;
  }
  // of sequence b
  __device__ __forceinline__ void find(const AttnArgs& a, int64_t b) {
    const int64_t g = group_of(a.prefix, b);
    take(a, g, g < 0 ? 0 : a.prefix.lens[g]);
  }
  // the same, each lane's own b, where the groups may be at hand; all lanes call it, as any of
  // them may have a group that others ask for
  __device__ __forceinline__ void find(const AttnArgs& a, int64_t b, const FirstGroups& groups) {
    if (a.prefix.n_seqs > 16) return find(a, b);
    take(a, -1, 0);
    for (int g = (int)a.prefix.n_seqs - 1; g >= 0; g--) {
      const int from = __builtin_amdgcn_readlane(groups.first, g), to = __builtin_amdgcn_readlane(groups.last, g);
      const int n = __builtin_amdgcn_readlane(groups.len, g);
      if (from <= b && b < to) take(a, g, n);
    }
  }
  __device__ __forceinline__ int tokens() const { return MODE == kBehind ? steps * kUnit : 0; }
  __device__ __forceinline__ bool has(int t) const { return MODE == kBehind && t < steps * kUnit; }
  // Of the tokens around position t: their end (`hi` that of the own ones), the row
  // of the table that has them, the position of its first token.
  __device__ __forceinline__ int end(int t, int hi) const { return has(t) ? len : hi; }
  __device__ __forceinline__ const int32_t* row(int t, const int32_t* own) const { return has(t) ? table : own; }
  __device__ __forceinline__ int origin(int t) const { return has(t) ? 0 : tokens(); }
  // the step at T has positions without a token
  __device__ __forceinline__ bool gap(int T) const { return MODE == kBehind && T + kUnit == steps * kUnit && len < steps * kUnit; }
  // end of the tokens that a row at position p of `n` sees
  __device__ __forceinline__ int sees_to(int causal, int p, int n) const {
    const int e = causal ? min(n, p + 1) : n;
    return MODE == kBehind ? max(e, steps * kUnit) : e;
  }
};

// Work items numbered in the order of the sequences, sequence b having
// count(b) of them: each thread sums a run of sequences, one scan joins them.
// Workgroups are numbered over the work that exists (the host only knows
// bounds): empty workgroups between full ones would not be spread evenly, as
// workgroups go to the shader engines in turn whether or not they have work.
template <int THREADS, class Count>
struct ItemScan {
  Count count;
  int64_t n_seqs, per, first, mine, total;  // this thread's run: its first item and their number
  int64_t* lds;                             // [THREADS / 64 + 2]

  // a batch of at most 64: every wave by itself, sequence b in lane b
  __device__ __forceinline__ bool few() const { return n_seqs <= 64; }

  __device__ __forceinline__ ItemScan(int64_t n, Count c, int64_t* mem) : count(c), n_seqs(n), lds(mem) {
    const int tid = threadIdx.x, lane = tid & 63, run = few() ? lane : tid;
    per = few() ? 1 : (n_seqs + THREADS - 1) / THREADS;
    mine = 0;
    for (int64_t b = run * per; b < min(n_seqs, (run + 1) * per); b++) mine += count(b);
    int64_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      if (few() && d >= n_seqs) break;
      const int64_t v = __shfl_up((long long)sum, d);
      sum += lane >= d ? v : 0;
    }
    int64_t before = 0;
    if (few()) {
      total = uniform64(__shfl((long long)sum, (int)n_seqs - 1));
    } else {
      if (lane == 63) lds[tid >> 6] = sum;
      __syncthreads();
      total = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 64; w++) {
        before += w < (tid >> 6) ? lds[w] : 0;
        total += lds[w];
      }
    }
    first = before + sum - mine;
  }
  // sequence and item in it of index k < total (the whole workgroup calls it)
  __device__ __forceinline__ void find(int64_t k, int64_t* b, int64_t* item) {
    if (few()) {
      const int at = __builtin_ctzll(__ballot(k >= first && k < first + mine));
      *b = at;
      *item = k - uniform64(__shfl((long long)first, at));
      return;
    }
    if (k >= first && k < first + mine) {
      int64_t i = threadIdx.x * per, left = k - first;
      for (;; i++) {
        const int64_t c = count(i);
        if (left < c) break;
        left -= c;
      }
      lds[THREADS / 64] = i;
      lds[THREADS / 64 + 1] = left;
    }
    __syncthreads();
    *b = uniform64(lds[THREADS / 64]);
    *item = uniform64(lds[THREADS / 64 + 1]);
    __syncthreads();
  }
};

// Few rows.  A tile is 16 NC rows of one sequence and key head, its work the
// blocks of 256 tokens (a step of 64 for each of the four waves) that any of
// them sees.  A fixed number of workgroups take equal, contiguous shares of all
// blocks of all tiles, or one block each where there are no more blocks; every
// wave reads the codes it needs straight from the cache into registers.  A tile
// that lies in several shares is joined by the workgroup that ends last.
// (Shares of single steps, which often had the end of one tile and the start of
// the next: 4 x 4 tokens in contexts of 777 23.1 us, with blocks 14.0 us; one
// token in 16000, D = 256, 28.1 and 23.4 us.)  Bound by memory: 32 tokens in
// ragged contexts up to 16384, 40 heads over 8, D = 128, 135 us (695 MB, 5.1
// TB/s); one in 131071, 24 heads over 4, D = 256, 65 us (268 MB, 4.1 TB/s; 57 us
// where the same cache was read just before and part of it lies in the last-level
// cache); 64 in 8192, 16 heads over 4, D = 64, 58 us (268 MB, 4.6 TB/s); one in 77, 40
// heads over 8, 8.3 us: start, one block a workgroup, the sums of the waves (10.0 us
// where the waves handed their O down in turn and one of them wrote all rows).
constexpr int kJoinLoads = 8;   // results of a pair of outputs read at once
constexpr int kMaxJoin = 32;    // results joined by one workgroup: shares of a tile <= kMaxJoin^2
constexpr int kMaxShares = 512;

// Parts of a tile of `steps` steps: at most the launch's, which knows only a
// bound on the length.  A step takes some 1.5 us, a part more to join 0.4: twice
// the root of the steps is best (40 tokens of 32 heads over 8, D = 128, in 4096
// tokens: 27 us in 32 parts, 22 in 16, 26 in 8; in 1024 16 us in 8, 19 in 4, 25
// in 2; in 1000 with a bound of 131072 36 us without this limit).
__device__ __forceinline__ int parts_of(int steps, int most) {
  return max(1, min((int)(2.f * __builtin_amdgcn_sqrtf((float)steps)), most));
}

// two floats, device-coherent
__device__ __forceinline__ void put2(float* p, float x, float y) {
  __hip_atomic_store((uint64_t*)p, (uint64_t)__float_as_uint(x) | ((uint64_t)__float_as_uint(y) << 32),
                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* p) {
  const uint64_t v = __hip_atomic_load((const uint64_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

// Four waves, so that two workgroups share a compute unit where a wave fits
// 256 registers and one starts or ends while the other reads.  D = 128 fills them; 96 to
// 116 scalars lie in lanes of vector registers, 131 to 159 of kBehind.
constexpr int kDecWaves = 4;
constexpr int kBlock = kUnit * kDecWaves;  // tokens of a block: a step of every wave

template <int D, int NC, int MODE>
__global__ __launch_bounds__(64 * kDecWaves, D * NC <= 128 ? 2 : 1) void attn_decode(AttnArgs a) {
  constexpr int DC = D / 64, DT = D / 16;
  __shared__ __attribute__((aligned(16))) float lo_[kDecWaves][NC * 16 * D];  // the waves' O
  __shared__ float lm_[kDecWaves][NC * 16], ll_[kDecWaves][NC * 16];
  __shared__ int64_t scan_[kDecWaves + 2];
  __shared__ uint32_t s_last;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int P = 1 << a.kv.lp;
  auto span_of = [&](int64_t i, Head<MODE>* head) -> SeqSpan {
    SeqSpan t = seq_span<MODE == kHead>(a.kv, i);
    if constexpr (MODE == kBehind || MODE == kTail) {
      head->find(a, i);
      t.len += head->tokens();
    }
    return t;
  };
  // a batch of at most 64 (not kPlain): read once, sequence b in lane b
  const bool near = MODE != kPlain && a.kv.n_seqs <= 64;
  SeqSpan mine = {0, 0, 0};
  Head<MODE> my_head;
  if (near) {
    FirstGroups groups;
    if constexpr (MODE == kBehind || MODE == kTail) groups.read(a.prefix);
    const int64_t b = min((int64_t)lane, a.kv.n_seqs - 1);
    mine = seq_span<MODE == kHead>(a.kv, b);
    if constexpr (MODE == kBehind || MODE == kTail) my_head.find(a, b, groups);
    mine.len += my_head.tokens();
  }
  auto span_for_all = [&](int64_t i, Head<MODE>* head) -> SeqSpan {
    if (!near) return span_of(i, head);
    SeqSpan t;
    t.row0 = uniform64(__shfl((long long)mine.row0, (int)i));
    t.n = __builtin_amdgcn_readlane(mine.n, (int)i);
    t.len = __builtin_amdgcn_readlane(mine.len, (int)i);
    if constexpr (MODE == kBehind || MODE == kTail)
      head->take(a, __builtin_amdgcn_readlane((int)my_head.group, (int)i), __builtin_amdgcn_readlane(my_head.len, (int)i));
    return t;
  };
  // blocks of one tile of a sequence (at least one, which writes its rows), and its tiles
  auto blocks_of = [&](const SeqSpan& t) -> int64_t {
    int64_t most = t.len;
    if (a.window > 0 && a.causal) most = min(most, (int64_t)a.window + t.n + kUnit);
    return max((most + kBlock - 1) / kBlock, (int64_t)1);
  };
  auto tiles_of = [&](const SeqSpan& t) -> int64_t { return (t.n * a.G + 16 * NC - 1) / (16 * NC); };
  // new token and head of row r of a sequence and key head (less than 2^31 rows, checked at the entry)
  const uint32_t G = (uint32_t)a.G;
  auto token_of = [&](int64_t r) -> int { return (int)((uint32_t)r / G); };
  auto head_of = [&](int64_t r) -> int { return (int)((uint32_t)r % G); };
  // kTail, and kBehind where a.pieces is set: a tile is cut into so many pieces at most, one
  // workgroup each (equal shares of all blocks would often have the end of one tile and the
  // start of the next)
  const int64_t pieces = MODE == kTail || MODE == kBehind ? a.pieces : 0;
  const bool in_pieces = MODE == kTail || (MODE == kBehind && pieces > 0);
  auto work_of = [&](int64_t i) -> int64_t {
    Head<MODE> head;
    const SeqSpan t = near ? mine : span_of(i, &head);  // near: i is the lane
    return tiles_of(t) * (in_pieces ? pieces : blocks_of(t));
  };
  ItemScan<64 * kDecWaves, decltype(work_of)> scan(a.kv.n_seqs, work_of, scan_);
  // in pieces: the tiles that the launch has workgroups for; starts that overlap could name more, and a
  // workgroup has one piece
  const int64_t per_head = scan.total, all = per_head * a.kv.H;
  const int64_t total = in_pieces ? min(all, quot(gridDim.x, pieces) * pieces) : all;
  // Shares: one for each block while there are workgroups for that, so that none
  // has parts of two tiles, which it would have to begin and join in turn
  const int64_t shares = max(min(total, (int64_t)gridDim.x), (int64_t)1);
  // Neighbouring shares on one XCD (bid % 8): where every workgroup has one; and pieces behind
  // prefixes, so that sequences of a group find its codes in their L2 (a grid of whole eights)
  const int64_t per_xcd = MODE == kBehind && in_pieces ? (shares + 7) / 8 : gridDim.x / 8, bid = blockIdx.x;
  int64_t share = bid;
  if (MODE == kBehind && in_pieces) {
    share = bid / 8 < per_xcd ? (bid % 8) * per_xcd + bid / 8 : shares;
  } else if (MODE != kTail && shares == (int64_t)gridDim.x) {
    share = (bid % 8) * per_xcd + bid / 8;
  }
  if (share >= shares) return;
  int64_t x = quot(total * share, shares);
  const int64_t x_end = quot(total * (share + 1), shares);
  if (x >= x_end) return;
  int h = (int)quot(x, per_head);
  int64_t b, item;
  scan.find(x - h * per_head, &b, &item);
  Head<MODE> head;
  SeqSpan s = span_for_all(b, &head);
  int64_t blocks = blocks_of(s), tiles = tiles_of(s);
  int64_t rt = quot(item, in_pieces ? pieces : blocks);
  int at = (int)(item - rt * (in_pieces ? pieces : blocks));  // first block of this share in the tile
  for (;;) {
    int count, n_parts;
    int64_t share0;  // the first share that holds blocks of this tile
    if (in_pieces) {
      n_parts = (int)min(pieces, blocks);
      share0 = share - at;
      if (at >= n_parts) return;
      const int first_block = (int)(blocks * at / n_parts);
      count = (int)(blocks * (at + 1) / n_parts) - first_block;
      at = first_block;
    } else {
      const int64_t x0 = x - at;  // the tile's first block among all
      count = (int)min(blocks - at, x_end - x);
      share0 = quot((x0 + 1) * shares + total - 1, total) - 1;
      n_parts = (int)(quot((x0 + blocks) * shares + total - 1, total) - 1 - share0 + 1);
    }
    const int64_t R = (int64_t)s.n * a.G;
    const int64_t rho0 = rt * 16 * NC;
    const int len = s.len, first = len - s.n;  // position of the first new token

    // visible tokens of this lane's rows: [vlo, vhi)
    int vlo[NC], vhi[NC];
    int hi_max = 0, hi_min = len, lo_min = 0, lo_max = 0;
    {
      const int64_t rlast = rho0 + 16 * NC - 1 < R ? rho0 + 16 * NC - 1 : R - 1;
      const int p0 = first + token_of(rho0), p1 = first + token_of(rlast);
      hi_max = head.sees_to(a.causal, p1, len);
      hi_min = head.sees_to(a.causal, p0, len);
      hi_max = max(hi_max, 0);
      hi_min = max(hi_min, 0);
      if (a.window > 0) {
        lo_min = max(0, p0 - a.window + 1);
        lo_max = max(0, p1 - a.window + 1);
      }
    }
    int64_t rho[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
      rho[c] = rho0 + 16 * c + n;
      const int64_t rc = rho[c] < R ? rho[c] : R - 1;
      const int p = first + token_of(rc);
      vhi[c] = head.sees_to(a.causal, p, len);
      vlo[c] = a.window > 0 ? max(0, p - a.window + 1) : 0;
    }
    const int u0 = lo_min / kUnit + kDecWaves * at, u1 = min(u0 + kDecWaves * count, (hi_max + kUnit - 1) / kUnit);

    // Q: lane (n, g) holds dims 64 c + 16 g + 8 e .. + 7 of its row
    v8bf qf[NC][DC][2];
#pragma unroll
    for (int c = 0; c < NC; c++) {
      const int64_t rc = rho[c] < R ? rho[c] : R - 1;
      const uint16_t* qp = a.q + (s.row0 + token_of(rc)) * a.q_stride + (h * a.G + head_of(rc)) * D + 16 * g;
#pragma unroll
      for (int d = 0; d < DC; d++) {
        qf[c][d][0] = __builtin_bit_cast(v8bf, *(const mx_u4*)(qp + 64 * d));
        qf[c][d][1] = __builtin_bit_cast(v8bf, *(const mx_u4*)(qp + 64 * d + 8));
      }
    }

    v4f o[NC][DT];
    float m[NC], l[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
      m[c] = -INFINITY;
      l[c] = 0.f;
#pragma unroll
      for (int d = 0; d < DT; d++) o[c][d] = v4f{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t* table = a.kv.table + b * a.kv.width;
    const int64_t page_bytes = ((int64_t)D << a.kv.lp);
    // Entry of the 16 tokens from t on, and the page it names: -1 where there are
    // none, -2 where it is unusable.  (Looked at when the page is needed: looked at
    // when read, it would be waited for, and every load before it.)
    auto entry_at = [&](int t) -> int {
      return head.row(t, table)[(min(t, head.end(t, hi_max) - 1) - head.origin(t)) >> a.kv.lp];
    };
    auto page_of = [&](int t, int entry) -> int {
      return t >= head.end(t, hi_max) ? -1 : entry >= 0 && entry < (int)a.kv.n_pages ? entry : -2;
    };
    mx_u4 kr[4][DC], vr[DT];
    int pgv = -1, pkn = 0, pvn = 0;  // this step's values' page, the next step's keys' and values' entries
    uint32_t kb = 0, vb = 0;           // exponent bytes of the lane's keys and values
    auto next_pages = [&](int u) {
      pkn = entry_at(u * kUnit + 16 * (n >> 2));
      pvn = entry_at(u * kUnit + 16 * g);
    };
    auto load_k = [&](int u) {
      const int tk = u * kUnit + 16 * (n >> 2);
      const int64_t ph = (int64_t)max(page_of(tk, pkn), 0) * a.kv.H + h;
      const uint8_t* kp = a.kv.kc + ph * page_bytes + (int64_t)(((tk - head.origin(tk)) & (P - 1)) + (n & 3)) * D + 16 * g;
      kb = a.kv.ks[ph];
#pragma unroll
      for (int t = 0; t < 4; t++)
#pragma unroll
        for (int d = 0; d < DC; d++) kr[t][d] = *(const mx_u4*)(kp + 4 * t * D + 64 * d);
    };
    auto load_v = [&](int u, int entry) {
      const int tv = u * kUnit + 16 * g;
      pgv = page_of(tv, entry);
      const int64_t ph = (int64_t)max(pgv, 0) * a.kv.H + h;
      const uint8_t* vp = a.kv.vc + ph * page_bytes + (int64_t)n * P + ((tv - head.origin(tv)) & (P - 1));
      vb = a.kv.vs[ph];
#pragma unroll
      for (int d = 0; d < DT; d++) vr[d] = *(const mx_u4*)(vp + (int64_t)16 * d * P);
    };

    // Loads in flight at any time: the next keys behind the scores of this step,
    // the next values behind its second product; page numbers a step earlier.
    int u = u0 + wave, pvu = 0;
    if (u < u1) {
      next_pages(u);
      pvu = pvn;
      load_k(u);
      if (u + kDecWaves < u1) next_pages(u + kDecWaves);
      load_v(u, pvu);
    }
    for (; u < u1; u += kDecWaves) {
      const bool gone = pgv < 0;  // none of this lane's 16 tokens can be read
      const float sk = pow2_byte(kb), sv = gone ? 0.f : pow2_byte(vb);
      if (pgv == -2 && n == 0 && a.kv.bad) atomicAdd(a.kv.bad, 1);
      const int T = u * kUnit;
      const bool part = T + kUnit > hi_min || T < lo_max || head.gap(T) || __any(gone);
      // scores of tokens T + 16 g + 4 t + j
      v4f sc[NC][4];
#pragma unroll
      for (int t = 0; t < 4; t++) {
#pragma unroll
        for (int c = 0; c < NC; c++) sc[c][t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < DC; d++) {
          const v8bf k0 = bf16x8_of_e4m3(kr[t][d].x, kr[t][d].y, sk), k1 = bf16x8_of_e4m3(kr[t][d].z, kr[t][d].w, sk);
#pragma unroll
          for (int c = 0; c < NC; c++) {
            sc[c][t] = mfma(k0, qf[c][d][0], sc[c][t]);
            sc[c][t] = mfma(k1, qf[c][d][1], sc[c][t]);
          }
        }
      }
      if (u + kDecWaves < u1) {
        load_k(u + kDecWaves);
        pvu = pvn;
        if (u + 2 * kDecWaves < u1) next_pages(u + 2 * kDecWaves);
      }
      v8bf pf[NC][2][2];  // weights in two bf16 terms
      uint32_t seen[NC];  // bit e: token 16 g + e is visible to the lane's row
#pragma unroll
      for (int c = 0; c < NC; c++) {
        float mx = -INFINITY;
        seen[c] = 0xFFFFu;
        if (part) {
          seen[c] = 0;
#pragma unroll
          for (int e = 0; e < 16; e++) {
            const int tok = T + 16 * g + e;
            const bool see = tok >= vlo[c] && tok < head.end(T, vhi[c]) && !gone;
            seen[c] |= see ? 1u << e : 0u;
            sc[c][e >> 2][e & 3] = see ? sc[c][e >> 2][e & 3] * a.scale2 : -INFINITY;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; e++) sc[c][e >> 2][e & 3] *= a.scale2;
        }
#pragma unroll
        for (int e = 0; e < 16; e++) mx = fmaxf(mx, sc[c][e >> 2][e & 3]);
        const float mn = fmaxf(m[c], group_max(mx));
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m[c] - mu);  // first tokens: 2^-inf = 0
        m[c] = mn;
        l[c] *= al;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
          for (int e = 0; e < 4; e++) o[c][d][e] *= al;
        float p[16];
#pragma unroll
        for (int e = 0; e < 16; e++) {
          p[e] = __builtin_amdgcn_exp2f(sc[c][e >> 2][e & 3] - mu);
          l[c] += p[e];
        }
#pragma unroll
        for (int e = 0; e < 16; e++) {
          const __bf16 hi = (__bf16)p[e];
          pf[c][e >> 3][0][e & 7] = hi;
          pf[c][e >> 3][1][e & 7] = (__bf16)(p[e] - (float)hi);
        }
      }
      if (part) {
        // Tokens no row sees: their codes may be anything, so they become 0.
        // A NaN code of a token that only some rows see must reach those rows
        // alone: it becomes 0 too and is put back below.
        uint32_t nans = 0;
        const int lo = (gone ? 16 : lo_min - (T + 16 * g)), hi = head.end(T, hi_max) - (T + 16 * g);
        const uint32_t k0 = byte_range(lo, hi), k1 = byte_range(lo - 4, hi - 4);
        const uint32_t k2 = byte_range(lo - 8, hi - 8), k3 = byte_range(lo - 12, hi - 12);
#pragma unroll
        for (int d = 0; d < DT; d++) {
          vr[d].x &= k0;
          vr[d].y &= k1;
          vr[d].z &= k2;
          vr[d].w &= k3;
          nans |= nan_bytes(vr[d].x) | nan_bytes(vr[d].y) | nan_bytes(vr[d].z) | nan_bytes(vr[d].w);
        }
        if (__any(nans != 0)) {
          v8bf vis[NC][2];
#pragma unroll
          for (int c = 0; c < NC; c++)
#pragma unroll
            for (int e = 0; e < 16; e++) vis[c][e >> 3][e & 7] = (__bf16)((seen[c] >> e) & 1u ? 1.0f : 0.0f);
#pragma unroll
          for (int d = 0; d < DT; d++) {
            v8bf isn[2];
#pragma unroll
            for (int e = 0; e < 16; e++) {
              const uint32_t w = (&vr[d])[0][e >> 2];
              isn[e >> 3][e & 7] = (__bf16)((nan_bytes(w) >> (8 * (e & 3) + 7)) & 1u ? 1.0f : 0.0f);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) vr[d][i] &= ~((nan_bytes(vr[d][i]) >> 7) * 0xFFu);
#pragma unroll
            for (int c = 0; c < NC; c++) {
              v4f hit = v4f{0.f, 0.f, 0.f, 0.f};
              hit = mfma(isn[0], vis[c][0], hit);
              hit = mfma(isn[1], vis[c][1], hit);
#pragma unroll
              for (int e = 0; e < 4; e++)
                if (hit[e] > 0.f) o[c][d][e] = __uint_as_float(0x7FC00000u);
            }
          }
        }
      }
#pragma unroll
      for (int d = 0; d < DT; d++) {
        const v8bf v0 = bf16x8_of_e4m3(vr[d].x, vr[d].y, sv), v1 = bf16x8_of_e4m3(vr[d].z, vr[d].w, sv);
#pragma unroll
        for (int c = 0; c < NC; c++) {
#pragma unroll
          for (int t = 0; t < 2; t++) {
            o[c][d] = mfma(v0, pf[c][0][t], o[c][d]);
            o[c][d] = mfma(v1, pf[c][1][t], o[c][d]);
          }
        }
      }
      if (u + kDecWaves < u1) load_v(u + kDecWaves, pvu);
    }

    if constexpr (MODE == kTail) {
      // The sums over the prefix: its parts for the waves of the tile's pieces in turn,
      // kTake of them on their way at once.
      constexpr int kTake = 4;
      const int parts = head.len > 0 ? parts_of(head.steps, a.sums_parts) : 0, takers = kDecWaves * n_parts;
#pragma unroll
      for (int c = 0; c < NC; c++) {
        const int64_t rc = rho[c] < R ? rho[c] : R - 1;
        const float* sums = a.sums + ((s.row0 + token_of(rc)) * a.Hq + h * a.G + head_of(rc)) * (D + kPartPad);
        const int64_t next = a.kv.total_q * a.Hq * (D + kPartPad);  // part
        for (int k = (int)(share - share0) * kDecWaves + wave; k < parts; k += takers * kTake) {
          float2 ml[kTake];
          v4f v[kTake][DT];
#pragma unroll
          for (int i = 0; i < kTake; i++) {
            const bool is = k + i * takers < parts;
            const float* from = sums + (is ? k + i * takers : k) * next;
            ml[i] = *(const float2*)(from + D);
            ml[i].x = is ? ml[i].x : -INFINITY;
#pragma unroll
            for (int d = 0; d < DT; d++) v[i][d] = *(const v4f*)(from + 16 * d + 4 * g);
          }
          float mn = m[c];
#pragma unroll
          for (int i = 0; i < kTake; i++) mn = fmaxf(mn, ml[i].x);
          const float mu = mn == -INFINITY ? 0.f : mn, al = __builtin_amdgcn_exp2f(m[c] - mu);
          m[c] = mn;
          l[c] *= al;
#pragma unroll
          for (int d = 0; d < DT; d++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[c][d][e] *= al;
#pragma unroll
          for (int i = 0; i < kTake; i++) {
            if (k + i * takers >= parts) break;
            const float w = __builtin_amdgcn_exp2f(ml[i].x - mu);
            l[c] += g == 0 ? w * ml[i].y : 0.f;  // the lanes of a row are added below
#pragma unroll
            for (int d = 0; d < DT; d++)
#pragma unroll
              for (int e = 0; e < 4; e++) o[c][d][e] += w * v[i][d][e];
          }
        }
      }
    }

    // ---- the waves' results: common maximum, then O added in the order of the waves
#pragma unroll
    for (int c = 0; c < NC; c++) {
      l[c] += __shfl_xor(l[c], 16);
      l[c] += __shfl_xor(l[c], 32);
      if (g == 0) {
        lm_[wave][16 * c + n] = m[c];
        ll_[wave][16 * c + n] = l[c];
      }
    }
    __syncthreads();
    // maximum and sum of weights of a row of the tile
    auto stats_of = [&](int row, float* mt, float* lt) {
      float mm = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWaves; w++) mm = fmaxf(mm, lm_[w][row]);
      const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
      for (int w = 0; w < kDecWaves; w++) L += ll_[w][row] * __builtin_amdgcn_exp2f(lm_[w][row] - mu);
      *mt = mm;
      *lt = L;
    };
#pragma unroll
    for (int c = 0; c < NC; c++) {
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kDecWaves; w++) mm = fmaxf(mm, lm_[w][16 * c + n]);
      const float f = __builtin_amdgcn_exp2f(m[c] - (mm == -INFINITY ? 0.f : mm));
#pragma unroll
      for (int d = 0; d < DT; d++) {
#pragma unroll
        for (int e = 0; e < 4; e++) o[c][d][e] *= f;
        *(v4f*)&lo_[wave][((c * DT + d) * 64 + lane) * 4] = o[c][d];
      }
    }
    __syncthreads();
    // every thread adds eight dims of a row, rows fastest: put(row, dims 8 q .., O)
    auto add_up = [&](int rows, auto&& put) {
      for (int i = threadIdx.x; i < NC * 2 * D; i += 64 * kDecWaves) {
        const int c = i / (2 * D), q = i / 16 % (D / 8), row = 16 * c + (i & 15);
        if (row >= rows) continue;
        const float* at = &lo_[0][((c * DT + q / 2) * 64 + 32 * (q & 1) + (i & 15)) * 4];
        v4f y[2];
#pragma unroll
        for (int k = 0; k < 2; k++) {
          v4f v[kDecWaves];
#pragma unroll
          for (int w = 0; w < kDecWaves; w++) v[w] = *(const v4f*)(at + w * (NC * 16 * D) + 64 * k);
#pragma unroll
          for (int e = 0; e < 4; e++) y[k][e] = (v[0][e] + v[2][e]) + (v[1][e] + v[3][e]);
        }
        put(row, q, y);
      }
    };
    static_assert(kDecWaves == 4, "the sum above");
    const int rows = (int)(R - rho0 < 16 * NC ? R - rho0 : 16 * NC);

    if (n_parts == 1) {
      add_up(rows, [&](int row, int q, const v4f* y) {
        float mt, lt;
        stats_of(row, &mt, &lt);
        const int64_t tok = s.row0 + token_of(rho0 + row), hd = h * a.G + head_of(rho0 + row);
        if constexpr (MODE == kHead) {
          float* sums = a.sums + (tok * a.Hq + hd) * (D + kPartPad);
          *(v4f*)(sums + 8 * q) = y[0];
          *(v4f*)(sums + 8 * q + 4) = y[1];
          if (q == 0) *(float2*)(sums + D) = make_float2(mt, lt);
          return;
        }
        const float inv = lt > 0.f || lt != lt ? 1.0f / lt : 0.f;
        mx_u4 w;
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] = bf16_bits(y[k / 2][2 * (k & 1)] * inv) | (bf16_bits(y[k / 2][2 * (k & 1) + 1] * inv) << 16);
        *(mx_u4*)(a.o + tok * a.o_stride + hd * D + 8 * q) = w;
        if (a.lse && q == 0) a.lse[tok * a.Hq + hd] = lt == 0.f ? -INFINITY : (mt + __builtin_amdgcn_logf(lt)) * kLn2;
      });
    } else {
      // ---- Several shares: results to the workspace with device-coherent stores
      // that complete before the arrival is counted.  A share has at most two
      // such tiles, so it has two places: 2 share for a tile that began in an
      // earlier one, 2 share + 1 for one that goes on.  Results are joined in the
      // order of the shares in groups, by the last of a group to arrive, then the
      // groups by the last of them: one workgroup reading every result of a long
      // context would take longer than reading the context.
      constexpr int PR = D + 2;                      // floats of one row: O, m, l
      constexpr int64_t PS = (int64_t)16 * NC * PR;  // of one place
      const int group = n_parts <= 64 ? 8 : kMaxJoin, groups = (n_parts + group - 1) / group;
      const int part_no = (int)(share - share0), grp = part_no / group;
      const int in_group = min(group, n_parts - grp * group);
      auto place = [&](int i) -> int64_t { return 2 * (share0 + i) + (i == 0 ? 1 : 0); };
      float* joined = a.part + 2 * (int64_t)kMaxShares * PS;  // a group's result, at the place of its first share
      uint32_t* group_cnt = a.cnt + place(grp * group);
      uint32_t* tile_cnt = a.cnt + 2 * kMaxShares + share0;
      add_up(rows, [&](int row, int q, const v4f* y) {
        float* to = a.part + place(part_no) * PS + row * PR;
#pragma unroll
        for (int k = 0; k < 4; k++) put2(to + 8 * q + 2 * k, y[k / 2][2 * (k & 1)], y[k / 2][2 * (k & 1) + 1]);
        if (q == 0) {
          float mt, lt;
          stats_of(row, &mt, &lt);
          put2(to + D, mt, lt);
        }
      });
      __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();  // every wave's stores are complete
      if (threadIdx.x == 0) s_last = __hip_atomic_fetch_add(group_cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      // in the LDS of the waves' results: [row][kMaxJoin] maxima, then weights; sums; joined m and l
      float* jw = &lo_[0][0];
      float* js = jw + 16 * NC * kMaxJoin;
      float* jm = js + 16 * NC * kMaxJoin;
      float* jl = jm + 16 * NC;
      static_assert(16 * NC * (2 * kMaxJoin + 2) <= kDecWaves * 16 * NC * D, "fits the waves' O");
      // joins the results at from(0 .. count - 1); each pair of outputs goes to put(row, dim, O, O)
      auto join = [&](auto&& from, int count, auto&& put) {
        for (int i = threadIdx.x; i < rows * count; i += 64 * kDecWaves) {
          const int r = i / count, k = i % count;
          const float2 v = get2(from(k) + r * PR + D);
          jw[r * kMaxJoin + k] = v.x;
          js[r * kMaxJoin + k] = v.y;
        }
        __syncthreads();
        if (threadIdx.x < rows) {
          const int r = threadIdx.x;
          float mm = -INFINITY, L = 0.f;
          for (int k = 0; k < count; k++) mm = fmaxf(mm, jw[r * kMaxJoin + k]);
          const float mu = mm == -INFINITY ? 0.f : mm;
          for (int k = 0; k < count; k++) {
            const float w = __builtin_amdgcn_exp2f(jw[r * kMaxJoin + k] - mu);
            L += w * js[r * kMaxJoin + k];
            jw[r * kMaxJoin + k] = w;
          }
          jm[r] = mm;
          jl[r] = L;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < rows * (D / 2); i += 64 * kDecWaves) {
          const int r = i / (D / 2), d = (i % (D / 2)) * 2;
          float px = 0.f, py = 0.f;
          for (int k0 = 0; k0 < count; k0 += kJoinLoads) {
            float2 v[kJoinLoads];
#pragma unroll
            for (int k = 0; k < kJoinLoads; k++)
              v[k] = k0 + k < count ? get2(from(k0 + k) + r * PR + d) : make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kJoinLoads; k++) {
              const float w = k0 + k < count ? jw[r * kMaxJoin + k0 + k] : 0.f;
              px += w * v[k].x;
              py += w * v[k].y;
            }
          }
          put(r, d, px, py);
        }
      };
      auto finish = [&](int r, int d, float px, float py) {
        const float L = jl[r], inv = L > 0.f || L != L ? 1.0f / L : 0.f;
        const int64_t tok = s.row0 + token_of(rho0 + r), hd = h * a.G + head_of(rho0 + r);
        if constexpr (MODE == kHead) {
          float* sums = a.sums + (tok * a.Hq + hd) * (D + kPartPad);
          *(float2*)(sums + d) = make_float2(px, py);
          if (d == 0) *(float2*)(sums + D) = make_float2(jm[r], L);
          return;
        }
        *(uint32_t*)(a.o + tok * a.o_stride + hd * D + d) = bf16_bits(px * inv) | (bf16_bits(py * inv) << 16);
        if (a.lse && d == 0) a.lse[tok * a.Hq + hd] = L == 0.f ? -INFINITY : (jm[r] + __builtin_amdgcn_logf(L)) * kLn2;
      };
      auto part_of_group = [&](int k) -> const float* { return a.part + place(grp * group + k) * PS; };
      if (s_last == (uint32_t)in_group - 1) {
        if (threadIdx.x == 0) __hip_atomic_store(group_cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (groups == 1) {
          join(part_of_group, n_parts, finish);
        } else {
          float* mine = joined + place(grp * group) * PS;
          join(part_of_group, in_group, [&](int r, int d, float px, float py) {
            put2(mine + r * PR + d, px, py);
            if (d == 0) put2(mine + r * PR + D, jm[r], jl[r]);
          });
          __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
          __syncthreads();  // every wave's stores are complete
          if (threadIdx.x == 0) s_last = __hip_atomic_fetch_add(tile_cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __syncthreads();
          if (s_last == (uint32_t)groups - 1) {
            if (threadIdx.x == 0) __hip_atomic_store(tile_cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            join([&](int k) -> const float* { return joined + place(k * group) * PS; }, groups, finish);
          }
        }
      }
    }
    // ---- the share's next tile
    x += in_pieces ? 1 : count;  // a share is one piece
    if (x >= x_end) return;
    __syncthreads();  // the LDS is free again
    at = 0;
    if (++rt == tiles) {
      rt = 0;
      do {
        if (++b == a.kv.n_seqs) {
          b = 0;
          h++;
        }
        s = span_for_all(b, &head);
        tiles = tiles_of(s);
      } while (tiles == 0);  // some sequence has tiles, as x < total
      blocks = blocks_of(s);
    }
  }
}

// ------------------------------------------------------------- many rows
// One workgroup per (sequence, key head, 16 NC WAVES rows).  A step's keys and
// values (64 tokens) are widened to bf16 once for all waves and lie in LDS as
// whole MFMA operands, 1 KiB per 16 rows x 32 k in the order of the lanes:
// writes and reads without bank conflicts.  2 x 4096 in 4096 tokens, causal, 24
// heads over 4, D = 256: 593 us (0.70 PFLOP/s).
// Where the tiles do not fill the chip, a tile's steps are cut into parts, one
// workgroup each, whose results attn_join puts together.
// steps [u0, u1) of part k of n
__device__ __forceinline__ void part_steps(int k, int n, int* u0, int* u1) {
  const int each = (*u1 - *u0) / n, more = (*u1 - *u0) - each * n;
  *u0 += each * k + min(k, more);
  *u1 = *u0 + each + (k < more ? 1 : 0);
}

// tokens that some of a run of rows see, [lo, hi), and that all of them see
struct Seen {
  int lo, hi, lo_all, hi_all;
};

// A workgroup's place in a prompt launch.
struct Place {
  int tile_at, h;  // tile of a head, and that
  int part, most;  // of the tile's steps, and as how many parts the launch has
  uint32_t slot;   // of its results in a.part
};
// heads run fastest, so that an XCD (bid % 8) keeps few of them in its L2
template <int MODE>
__device__ __forceinline__ Place place_of(const AttnArgs& a) {
  Place p;
  const uint32_t H = (uint32_t)a.kv.H, at = blockIdx.x / H, parts = (uint32_t)a.parts;
  p.h = (int)(blockIdx.x - at * H);
  const uint32_t whole = MODE == kBehind ? (uint32_t)a.whole : 0u;
  if (MODE == kBehind && at < whole) {
    p.tile_at = (int)at;
    p.part = 0;
    p.most = 1;
    p.slot = 0;
  } else {
    const uint32_t cut = (at - whole) / parts;
    p.tile_at = (int)(whole + cut);
    p.part = (int)(at - whole - cut * parts);
    p.most = a.parts;
    p.slot = blockIdx.x - whole * H;
  }
  return p;
}

// A tile of ROWS rows of one sequence and key head.
template <int ROWS, int MODE>
struct PromptTile {
  int64_t b;     // sequence
  SeqSpan s;
  int R, wg0;    // rows of the sequence and head (less than 2^31, checked at the entry), first of the tile
  int first;     // position of the first new token
  Seen seen;     // by the tile
  int u0, u1;    // steps of 64 tokens that some row sees
  int parts;     // they are cut into
  Head<MODE> head;

  // tile number `at` of a head, all sequences in turn, in at most `most` parts; false behind the last
  template <int THREADS>
  __device__ __forceinline__ bool find(const AttnArgs& a, uint32_t at, int most, int64_t* mem) {
    auto tiles = [&](int64_t i) -> int64_t { return (seq_span<MODE == kHead>(a.kv, i).n * a.G + ROWS - 1) / ROWS; };
    ItemScan<THREADS, decltype(tiles)> scan(a.kv.n_seqs, tiles, mem);
    if (at >= scan.total) return false;
    int64_t item;
    scan.find(at, &b, &item);
    s = seq_span<MODE == kHead>(a.kv, b);
    if constexpr (MODE == kBehind) {
      head.find(a, b);
      s.len += head.tokens();
    }
    R = s.n * (int)a.G;
    wg0 = (R - 1) / ROWS * ROWS - (int)item * ROWS;  // the last, longest tiles of a sequence first
    first = s.len - s.n;
    seen = of_rows(a, wg0, wg0 + ROWS);
    u0 = seen.lo / kUnit;
    u1 = (seen.hi + kUnit - 1) / kUnit;
    parts = parts_of(u1 - u0, most);
    return true;
  }
  __device__ __forceinline__ Seen of_rows(const AttnArgs& a, int r0, int r1) const {
    r0 = r0 < R - 1 ? r0 : R - 1;
    r1 = r1 < R ? r1 : R;
    const int p0 = first + (int)((uint32_t)r0 / (uint32_t)a.G), p1 = first + (int)((uint32_t)(r1 - 1) / (uint32_t)a.G);
    Seen v;
    v.hi = max(0, head.sees_to(a.causal, p1, s.len));
    v.hi_all = max(0, head.sees_to(a.causal, p0, s.len));
    v.lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    v.lo_all = a.window > 0 ? max(0, p1 - a.window + 1) : 0;
    return v;
  }
};

template <int D, int NC, int WAVES, int MODE, bool FINE>
__global__ __launch_bounds__(64 * WAVES, 2) void attn_prompt(AttnArgs a) {
  constexpr int DS = D / 32, DT = D / 16, HALF = 32 * WAVES, SP = 4 * D / HALF;
  static_assert(SP * HALF == 4 * D, "whole 16-byte pieces per thread");
  __shared__ __attribute__((aligned(16))) uint8_t k_[2][4 * DS * 1024], v_[2][DT * 2048];
  __shared__ int nan_at_[4];  // steps whose values hold NaN codes that were put aside
  const bool keys = __builtin_amdgcn_readfirstlane((int)threadIdx.x) < HALF;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  constexpr int ROWS = 16 * NC * WAVES;
  const Place at_ = place_of<MODE>(a);
  const uint32_t G = (uint32_t)a.G;
  const int h = at_.h, part = at_.part;
  __shared__ int64_t scan_[WAVES + 2];
  PromptTile<ROWS, MODE> t;
  if (!t.template find<64 * WAVES>(a, at_.tile_at, at_.most, scan_) || part >= t.parts) return;
  const SeqSpan s = t.s;
  const Head<MODE> head = t.head;
  const int R = t.R, wg0 = t.wg0, len = s.len, first = t.first, P = 1 << a.kv.lp, rho0 = wg0 + wave * 16 * NC;
  const int lo_min = t.seen.lo, hi_max = t.seen.hi, lo_all = t.seen.lo_all, hi_all = t.seen.hi_all;
  const Seen mine = t.of_rows(a, rho0, rho0 + 16 * NC);  // by this wave's rows
  const int wlo = mine.lo, wlo_all = mine.lo_all, whi_all = mine.hi_all;
  const int whi = __builtin_amdgcn_readfirstlane(rho0 < R ? mine.hi : 0);
  const bool none = a.scale2 == 0.f;  // all scores 0, or NaN
  int rho[NC], vlo[NC], vhi[NC];
  v8bf qf[NC][DS];
#pragma unroll
  for (int c = 0; c < NC; c++) {
    rho[c] = rho0 + 16 * c + n;
    const uint32_t rc = rho[c] < R ? rho[c] : R - 1, at = rc / G;
    const int p = first + (int)at;
    vhi[c] = head.sees_to(a.causal, p, len);
    vlo[c] = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const uint16_t* qp = a.q + (s.row0 + at) * a.q_stride + ((int64_t)h * G + (rc - at * G)) * D + 16 * g;
#pragma unroll
    for (int d = 0; d < DS; d++) {  // dims 64 (d / 2) + 16 g + 8 (d % 2) .. + 7
      mx_u4 w = *(const mx_u4*)(qp + 64 * (d >> 1) + 8 * (d & 1));
      // the maximum and the mask's -infinity below want a positive scale
      if (a.scale2 < 0.f) w ^= 0x80008000u;
      if (none) w = zero_or_nan(w);
      qf[c][d] = __builtin_bit_cast(v8bf, w);
    }
  }
  const float scale = none ? 1.f : fabsf(a.scale2);
  v4f o[NC][DT];
  float m[NC], l[NC];
  uint64_t nanned[NC];  // bit 4 d + e: o[c][d][e] meets a NaN value
#pragma unroll
  for (int c = 0; c < NC; c++) {
    m[c] = -INFINITY;
    l[c] = 0.f;
    nanned[c] = 0;
#pragma unroll
    for (int d = 0; d < DT; d++) o[c][d] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  const int parts = t.parts;
  int u0 = t.u0, u1 = t.u1;
  part_steps(part, parts, &u0, &u1);
  const int32_t* table = a.kv.table + t.b * a.kv.width;
  // Page of the 16 tokens that the lane stages from: tokens 64 u + 16 x .. with
  // x = row / 4 of the keys' operand, x = group of the values'.
  const int stage_group = keys ? (lane >> 2) & 3 : g;
  // their table entry, and the page it names: -1 where there are none, -2 where it
  // is unusable (looked at a step later: looked at when read, it would be waited for)
  auto entry_at = [&](int u) -> int {
    const int T = u * kUnit;
    return head.row(T, table)[(min(T + 16 * stage_group, head.end(T, hi_max) - 1) - head.origin(T)) >> a.kv.lp];
  };
  auto page_of = [&](int u, int entry) -> int {
    return u * kUnit + 16 * stage_group >= head.end(u * kUnit, hi_max) ? -1 : entry >= 0 && entry < (int)a.kv.n_pages ? entry : -2;
  };
  // This thread's 16-byte pieces of a step: of the keys for the first half of
  // the waves (wave t: the rows of tile t, piece i: dims 64 i + 16 g ..), of the
  // values for the second (16 tokens of dim 16 (t + 4 i) + n).  A wave's piece
  // makes two whole operands, lane by lane.
  mx_u4 raw[SP];
  uint32_t eb = 0;
  const int sh = a.kv.lp + (D == 64 ? 6 : D == 128 ? 7 : 8);  // log2 of a page's bytes of one head
  const int w4 = wave & (WAVES / 2 - 1);
  // row 4 g' + j of tile t is token 16 g' + 4 t + j
  const int tok = 16 * stage_group + 4 * w4 + (lane & 3);
  const uint32_t kat = (uint32_t)((tok & (P - 1)) * D + 16 * g);
  const uint32_t vat = (uint32_t)((16 * w4 + n) * P + ((16 * g) & (P - 1)));
  auto fetch = [&](int u, int pg) {
    const uint32_t in = (u * kUnit - head.origin(u * kUnit)) & (P - 1);  // the step's place in a larger page
    const int64_t ph = (int64_t)(pg < 0 ? 0 : pg) * a.kv.H + h;
    if (keys) {
      const uint8_t* kp = a.kv.kc + (ph << sh) + (kat + in * D);
      eb = a.kv.ks[ph];
#pragma unroll
      for (int i = 0; i < SP; i++) raw[i] = *(const mx_u4*)(kp + 64 * i);
    } else {
      const uint8_t* vp = a.kv.vc + (ph << sh) + (vat + in);
      eb = a.kv.vs[ph];
#pragma unroll
      for (int i = 0; i < SP; i++) raw[i] = *(const mx_u4*)(vp + (uint32_t)(64 * i * P));
    }
  };
  // tokens some row of the workgroup does not see, or that cannot be read
  auto partial = [&](int u, int pg) {
    return u * kUnit + kUnit > hi_all || u * kUnit < lo_all || head.gap(u * kUnit) || __any(pg < 0);
  };
  // widened and written to the step's buffer
  auto stage = [&](int u, int pg) {
    if (keys) {
      const float sc = pow2_byte(eb);
      uint8_t* w = k_[(u - u0) & 1] + w4 * DS * 1024 + 16 * lane;
#pragma unroll
      for (int i = 0; i < SP; i++) {
        *(v8bf*)(w + 2 * i * 1024) = bf16x8_of_e4m3(raw[i].x, raw[i].y, sc);
        *(v8bf*)(w + (2 * i + 1) * 1024) = bf16x8_of_e4m3(raw[i].z, raw[i].w, sc);
      }
    } else {
      const bool part = partial(u, pg);
      const float sc = pg < 0 ? 0.f : pow2_byte(eb);
      if (part) {
        // codes of tokens no row sees become 0; NaN codes too, and are put
        // back beside the products for the rows that see them
        const int T = u * kUnit + 16 * g, lo = pg < 0 ? 16 : lo_min - T, hi = head.end(u * kUnit, hi_max) - T;
        uint32_t nans = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint32_t keep = byte_range(lo - 4 * e, hi - 4 * e);
#pragma unroll
          for (int i = 0; i < SP; i++) {
            raw[i][e] &= keep;
            const uint32_t nb = nan_bytes(raw[i][e]);
            nans |= nb;
            raw[i][e] &= ~((nb >> 7) * 0xFFu);
          }
        }
        if (nans) nan_at_[u & 3] = u;
        if (pg == -2 && w4 == 0 && n == 0 && a.kv.bad) atomicAdd(a.kv.bad, 1);
      }
      uint8_t* w = v_[(u - u0) & 1] + w4 * 2048 + 16 * lane;
#pragma unroll
      for (int i = 0; i < SP; i++) {
        *(v8bf*)(w + i * 8192) = bf16x8_of_e4m3(raw[i].x, raw[i].y, sc);
        *(v8bf*)(w + i * 8192 + 1024) = bf16x8_of_e4m3(raw[i].z, raw[i].w, sc);
      }
    }
  };
  auto meet = [&]() {  // LDS reads and writes are done; loads stay in flight
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
  };

  const int at = 16 * lane;
  v4f sc[NC][4];
  v8bf pf[NC][2], pl[FINE ? NC : 1][2];  // weights; FINE: and what their rounding left
  auto sees = [&](int u) { return u * kUnit < whi && u * kUnit + kUnit > wlo; };
  // scores of step u
  auto scores = [&](int u) {
    const uint8_t* buf = k_[(u - u0) & 1];
    v8bf kf[2][DS];  // two tiles, so that four chains of products alternate
#pragma unroll
    for (int t = 0; t < 4; t += 2) {
#pragma unroll
      for (int d = 0; d < DS; d++)
#pragma unroll
        for (int e = 0; e < 2; e++) kf[e][d] = *(const v8bf*)(buf + ((t + e) * DS + d) * 1024 + at);
#pragma unroll
      for (int e = 0; e < 2; e++)
#pragma unroll
        for (int c = 0; c < NC; c++) sc[c][t + e] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < DS; d++)
#pragma unroll
        for (int e = 0; e < 2; e++)
#pragma unroll
          for (int c = 0; c < NC; c++) sc[c][t + e] = mfma(kf[e][d], qf[c][d], sc[c][t + e]);
    }
  };
  // O += P V of step u
  auto weigh = [&](int u) {
    const uint8_t* buf = v_[(u - u0) & 1];
    if (nan_at_[u & 3] == u) {
      // rare: a NaN code among tokens that not every row of the workgroup sees
      const int T = u * kUnit, vp = __shfl(page_of(u, entry_at(u)), keys ? 4 * g : lane);
      const uint8_t* vc = a.kv.vc + (((int64_t)(vp < 0 ? 0 : vp) * a.kv.H + h) << sh) + ((T + 16 * g - head.origin(u * kUnit)) & (P - 1));
#pragma unroll 1
      for (int d = 0; d < DT; d++) {
        const mx_u4 w = *(const mx_u4*)(vc + (int64_t)(16 * d + n) * P);
        v8bf isn[2];
#pragma unroll
        for (int e = 0; e < 16; e++)
          isn[e >> 3][e & 7] = (__bf16)(vp >= 0 && ((nan_bytes(w[e >> 2]) >> (8 * (e & 3) + 7)) & 1u) ? 1.f : 0.f);
#pragma unroll
        for (int c = 0; c < NC; c++) {
          v8bf vis[2];
#pragma unroll
          for (int e = 0; e < 16; e++) {
            const int tok = T + 16 * g + e;
            vis[e >> 3][e & 7] = (__bf16)(tok >= vlo[c] && tok < head.end(u * kUnit, vhi[c]) ? 1.f : 0.f);
          }
          v4f hit = v4f{0.f, 0.f, 0.f, 0.f};
          hit = mfma(isn[0], vis[0], hit);
          hit = mfma(isn[1], vis[1], hit);
#pragma unroll
          for (int e = 0; e < 4; e++) nanned[c] |= hit[e] > 0.f ? uint64_t(1) << (4 * d + e) : 0;
        }
      }
    }
    v8bf vf[2][4];
    auto read_v = [&](int d) {  // two tiles of 16 dims
#pragma unroll
      for (int e = 0; e < 4; e++) vf[(d >> 1) & 1][e] = *(const v8bf*)(buf + d * 2048 + e * 1024 + at);
    };
    read_v(0);
#pragma unroll
    for (int d = 0; d < DT; d += 2) {
      if (d + 2 < DT) read_v(d + 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = 0; f < 2; f++)
#pragma unroll
        for (int e = f; e < 4; e += 2)
#pragma unroll
          for (int c = 0; c < NC; c++) {
            o[c][d + (e >> 1)] = mfma(vf[(d >> 1) & 1][e], pf[c][f], o[c][d + (e >> 1)]);
            if constexpr (FINE) o[c][d + (e >> 1)] = mfma(vf[(d >> 1) & 1][e], pl[c][f], o[c][d + (e >> 1)]);
          }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // weights of step u from its scores
  auto softmax = [&](int u, int pg) {
    const int T = u * kUnit;
    const bool mask = T + kUnit > whi_all || T < wlo_all || head.gap(u * kUnit) || __any(pg < 0);
    const int page = mask ? __shfl(pg, keys ? 4 * g : lane) : 0;  // of the lane's 16 tokens
#pragma unroll
    for (int c = 0; c < NC; c++) {
      if (mask) {
        const int lo = page < 0 ? 16 : vlo[c] - (T + 16 * g), hi = head.end(u * kUnit, vhi[c]) - (T + 16 * g);
        const uint32_t up = hi >= 16 ? 0xFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
        const uint32_t seen = lo >= 16 ? 0u : lo <= 0 ? up : up & ~((1u << lo) - 1u);
#pragma unroll
        for (int e = 0; e < 16; e++) sc[c][e >> 2][e & 3] = (seen >> e) & 1u ? sc[c][e >> 2][e & 3] : -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 16; e++) mx = fmaxf(mx, sc[c][e >> 2][e & 3]);
      mx = group_max(mx) * scale;
      // The maximum in use may lag by up to 2^8 (weights up to 256 lose no
      // precision), so O is rescaled in few of the steps.
      if (__any(mx > m[c] + 8.f)) {
        const float mn = fmaxf(m[c], mx), mu = mn == -INFINITY ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m[c] - mu);  // first tokens: 2^-inf = 0
        m[c] = mn;
        l[c] *= al;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
          for (int e = 0; e < 4; e++) o[c][d][e] *= al;
      }
      const float mu = m[c] == -INFINITY ? 0.f : m[c];
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 16; e++) {
        const float p = __builtin_amdgcn_exp2f(fmaf(sc[c][e >> 2][e & 3], scale, -mu));  // masked: 2^-inf = 0
        sum[e & 3] += p;
        const __bf16 hi = (__bf16)p;
        pf[c][e >> 3][e & 7] = hi;
        if constexpr (FINE) pl[c][e >> 3][e & 7] = (__bf16)(p - (float)hi);
      }
      l[c] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
  };

  // Two phases a step: products (scores of step u, weighted values of u - 1),
  // then softmax and staging.  The second half of the waves runs one phase
  // behind the first, so that on every SIMD one wave multiplies while another
  // computes weights.  The first half stages the keys of u + 1, read from its
  // next phase on; the second the values of u + 1, read two steps on; either
  // buffer's last reader is a phase before.
  if (tid < 4) nan_at_[tid] = -1;
  __syncthreads();
  const int e0 = u0 < u1 ? entry_at(u0) : -1, e1 = u0 + 1 < u1 ? entry_at(u0 + 1) : -1;
  int pg0 = page_of(u0, e0), pg1 = page_of(u0 + 1, e1);
  if (u0 < u1) {
    fetch(u0, pg0);
    stage(u0, pg0);
  }
  meet();
  if (!keys) meet();
  for (int u = u0; u <= u1; u++) {
    const bool more = u + 1 < u1;
    const int e2 = u + 2 < u1 ? entry_at(u + 2) : -1;
    if (more) fetch(u + 1, pg1);
    if (u < u1 && sees(u)) scores(u);
    if (u > u0 && sees(u - 1)) weigh(u - 1);
    meet();
    if (u < u1 && sees(u)) softmax(u, pg0);
    if (more) stage(u + 1, pg1);
    pg0 = pg1;
    pg1 = page_of(u + 2, e2);
    if (keys || u < u1) meet();
  }
#pragma unroll
  for (int c = 0; c < NC; c++) {
    l[c] += __shfl_xor(l[c], 16);
    l[c] += __shfl_xor(l[c], 32);
    if (rho[c] >= R) continue;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 4; e++)
        if ((nanned[c] >> (4 * d + e)) & 1) o[c][d][e] = __uint_as_float(0x7FC00000u);
    const uint32_t tok = (uint32_t)rho[c] / G;
    const int64_t row = s.row0 + tok, hd = (int64_t)h * G + (rho[c] - tok * G);
    if (MODE == kHead || parts > 1) {
      float* pp = MODE == kHead ? a.sums + ((part * a.kv.total_q + row) * a.Hq + hd) * (D + kPartPad)
                                : a.part + ((int64_t)at_.slot * ROWS + (rho[c] - wg0)) * (D + kPartPad);
#pragma unroll
      for (int d = 0; d < DT; d++) *(v4f*)(pp + 16 * d + 4 * g) = o[c][d];
      if (g == 0) *(float2*)(pp + D) = make_float2(m[c], l[c]);
      continue;
    }
    const float inv = l[c] > 0.f || l[c] != l[c] ? 1.0f / l[c] : 0.f;
    uint16_t* op = a.o + row * a.o_stride + hd * D + 4 * g;
#pragma unroll
    for (int d = 0; d < DT; d++) {
      uint2 w;
      w.x = bf16_bits(o[c][d][0] * inv) | (bf16_bits(o[c][d][1] * inv) << 16);
      w.y = bf16_bits(o[c][d][2] * inv) | (bf16_bits(o[c][d][3] * inv) << 16);
      *(uint2*)(op + 16 * d) = w;
    }
    if (a.lse && g == 0) a.lse[row * a.Hq + hd] = l[c] == 0.f ? -INFINITY : (m[c] + __builtin_amdgcn_logf(l[c])) * kLn2;
  }
}

// The same for heads of 64 and 128 with 32 x 32 x 16 products: half the operand
// reads for a product, one row a lane, and products and multiply-adds of two
// waves of a SIMD overlap better (side by side they took 1 / 1.92 of their
// times' sum, with 16 x 16 x 32 products 1 / 1.66).  Row 8 x + 4 h + j of a tile
// of 32 tokens is token 16 h + 4 x + j, so that lane half h holds 16
// consecutive tokens.  2 prompts of 4096 in 4096 tokens, 40 heads over 8, all
// pairs: D = 128 801 -> 753 us.  4096 rows over 8192 tokens take 1453 us (0.95
// PFLOP/s) and 1212 us where all codes are 0, so power bounds much of it;
// products that begin with their operands read ahead across the phases took the
// same time, and weights without their exponentials 98%.  D = 64, causal: 342 us
// with 16 x 16 products, 315 us with 8 waves, 266 us with 4 waves and three
// workgroups a compute unit: more waves hide latency.  Its products keep the MFMA
// busy in 24% of the cycles, LDS is active in 20%; vector instructions take 47% at
// four cycles each and the exponentials' quarter rate some 17% more (2 x 4096 in
// 4096, 32 heads over 8: 226 us).  One register is spilled (kBehind: two).
template <int D, int NC, int WAVES, int OCC, int MODE, bool FINE>
__global__ __launch_bounds__(64 * WAVES, OCC) void attn_prompt32(AttnArgs a) {
  constexpr int DS = D / 16, DT = D / 32, HALF = 32 * WAVES, SP = 4 * D / HALF, PS = WAVES / 4;
  static_assert(SP * HALF == 4 * D, "whole 16-byte pieces per thread");
  constexpr int KB = 2 * DS * 1024, VB = 4 * DT * 1024;  // bytes of a step's operands
  constexpr int OUT = 2 * D + 16;                        // a row of O on its way out, padded against bank conflicts
  __shared__ __attribute__((aligned(16))) uint8_t lds_[2 * (KB + VB) > 32 * NC * WAVES * OUT ? 2 * (KB + VB) : 32 * NC * WAVES * OUT];
  // steps whose values hold NaN codes that were put aside; that name pages that cannot be read
  __shared__ int nan_at_[4], bad_at_[4];
  const bool keys = __builtin_amdgcn_readfirstlane((int)threadIdx.x) < HALF;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, hf = lane >> 5;
  constexpr int ROWS = 32 * NC * WAVES;
  const Place at_ = place_of<MODE>(a);
  const uint32_t G = (uint32_t)a.G;
  const int h = at_.h, part = at_.part;
  __shared__ int64_t scan_[WAVES + 2];
  PromptTile<ROWS, MODE> t;
  if (!t.template find<64 * WAVES>(a, at_.tile_at, at_.most, scan_) || part >= t.parts) return;
  const SeqSpan s = t.s;
  const Head<MODE> head = t.head;
  const int R = t.R, wg0 = t.wg0, len = s.len, first = t.first, P = 1 << a.kv.lp, rho0 = wg0 + wave * 32 * NC;
  const int lo_min = t.seen.lo, hi_max = t.seen.hi, lo_all = t.seen.lo_all, hi_all = t.seen.hi_all;
  const Seen mine = t.of_rows(a, rho0, rho0 + 32 * NC);  // by this wave's rows
  const int wlo = mine.lo, wlo_all = mine.lo_all, whi_all = mine.hi_all;
  const int whi = __builtin_amdgcn_readfirstlane(rho0 < R ? mine.hi : 0);
  const bool none = a.scale2 == 0.f;  // all scores 0, or NaN
  int rho[NC], vlo[NC], vhi[NC];
  v8bf qf[NC][DS];
#pragma unroll
  for (int c = 0; c < NC; c++) {
    rho[c] = rho0 + 32 * c + n;
    const uint32_t rc = rho[c] < R ? rho[c] : R - 1, at = rc / G;
    const int p = first + (int)at;
    vhi[c] = head.sees_to(a.causal, p, len);
    vlo[c] = a.window > 0 ? max(0, p - a.window + 1) : 0;
    const uint16_t* qp = a.q + (s.row0 + at) * a.q_stride + ((int64_t)h * G + (rc - at * G)) * D + 8 * hf;
#pragma unroll
    for (int d = 0; d < DS; d++) qf[c][d] = __builtin_bit_cast(v8bf, *(const mx_u4*)(qp + 16 * d));  // dims 16 d + 8 h .. + 7
  }
  const float scale = none ? 1.f : fabsf(a.scale2);
  v16f o[NC][DT];
  float m[NC], l[NC];
  uint64_t nanned[NC];  // bit 16 d + e: o[c][d][e] meets a NaN value
#pragma unroll
  for (int c = 0; c < NC; c++) {
    m[c] = -INFINITY;
    l[c] = 0.f;
    nanned[c] = 0;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int e = 0; e < 16; e++) o[c][d][e] = 0.f;
  }

  const int parts = t.parts;
  int u0 = t.u0, u1 = t.u1;
  part_steps(part, parts, &u0, &u1);
  const int32_t* table = a.kv.table + t.b * a.kv.width;
  // This thread's 16-byte pieces of a step.  Keys (first half of the waves,
  // tile w4 % 2): 16 dims 16 (2 (w4 / 2 + 2 i) + h) .. of the token of row n.
  // Values (second half): 16 tokens of dim 32 (w4 / 2 + 2 i) + n, tokens
  // 32 (w4 % 2) + 16 h ...  A piece of values is two operands lane by lane, of
  // keys the two halves of one.
  const int w4 = wave & (WAVES / 2 - 1), tile = w4 & 1;
  const int stage_group = 2 * tile + (keys ? (lane >> 2) & 1 : hf);  // of 16 tokens
  // their table entry, and the page it names: -1 where there are none, -2 where it
  // is unusable (looked at a step later: looked at when read, it would be waited for)
  auto entry_at = [&](int u) -> int {
    const int T = u * kUnit;
    return head.row(T, table)[(min(T + 16 * stage_group, head.end(T, hi_max) - 1) - head.origin(T)) >> a.kv.lp];
  };
  auto page_of = [&](int u, int entry) -> int {
    return u * kUnit + 16 * stage_group >= head.end(u * kUnit, hi_max) ? -1 : entry >= 0 && entry < (int)a.kv.n_pages ? entry : -2;
  };
  mx_u4 raw[SP];
  uint32_t eb = 0;
  const int sh = a.kv.lp + (D == 64 ? 6 : 7);  // log2 of a page's bytes of one head
  const int tok = 16 * stage_group + 4 * (n >> 3) + (n & 3);
  const uint32_t kat = (uint32_t)((tok & (P - 1)) * D + 32 * (w4 >> 1) + 16 * hf);
  const uint32_t vat = (uint32_t)((32 * (w4 >> 1) + n) * P + ((16 * stage_group) & (P - 1)));
  auto fetch = [&](int u, int pg) {
    const uint32_t in = (u * kUnit - head.origin(u * kUnit)) & (P - 1);  // the step's place in a larger page
    const int64_t ph = (int64_t)(pg < 0 ? 0 : pg) * a.kv.H + h;
    if (keys) {
      const uint8_t* kp = a.kv.kc + (ph << sh) + (kat + in * D);
      eb = a.kv.ks[ph];
#pragma unroll
      for (int i = 0; i < SP; i++) raw[i] = *(const mx_u4*)(kp + 32 * PS * i);
    } else {
      const uint8_t* vp = a.kv.vc + (ph << sh) + (vat + in);
      eb = a.kv.vs[ph];
#pragma unroll
      for (int i = 0; i < SP; i++) raw[i] = *(const mx_u4*)(vp + (uint32_t)(32 * PS * i * P));
    }
  };
  // tokens some row of the workgroup does not see, or that cannot be read
  auto partial = [&](int u, int pg) {
    return u * kUnit + kUnit > hi_all || u * kUnit < lo_all || head.gap(u * kUnit) || __any(pg < 0);
  };
  // widened and written to the step's buffer
  auto stage = [&](int u, int pg) {
    if (keys) {
      const float sc = pow2_byte(eb);
      // operand (tile, 16-dim block x): lane (n, half of the dims)
      uint8_t* w = lds_ + ((u - u0) & 1) * KB + (tile * DS + 2 * (w4 >> 1) + hf) * 1024 + 16 * n;
#pragma unroll
      for (int i = 0; i < SP; i++) {
        *(v8bf*)(w + 2 * PS * i * 1024) = bf16x8_of_e4m3(raw[i].x, raw[i].y, sc);
        *(v8bf*)(w + 2 * PS * i * 1024 + 512) = bf16x8_of_e4m3(raw[i].z, raw[i].w, sc);
      }
    } else {
      const bool part = partial(u, pg);
      const float sc = pg < 0 ? 0.f : pow2_byte(eb);
      if (part) {
        // codes of tokens no row sees become 0; NaN codes too, and are put
        // back beside the products for the rows that see them
        const int T = u * kUnit + 16 * stage_group, lo = pg < 0 ? 16 : lo_min - T, hi = head.end(u * kUnit, hi_max) - T;
        uint32_t nans = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint32_t keep = byte_range(lo - 4 * e, hi - 4 * e);
#pragma unroll
          for (int i = 0; i < SP; i++) {
            raw[i][e] &= keep;
            const uint32_t nb = nan_bytes(raw[i][e]);
            nans |= nb;
            raw[i][e] &= ~((nb >> 7) * 0xFFu);
          }
        }
        if (nans) nan_at_[u & 3] = u;
        if (pg == -2) bad_at_[u & 3] = u;
        if (pg == -2 && w4 < 2 && n == 0 && a.kv.bad) atomicAdd(a.kv.bad, 1);
      }
      // operand (16-token block x of 4: tile, 8 tokens; 32-dim tile): lane (n, h)
      uint8_t* w = lds_ + 2 * KB + ((u - u0) & 1) * VB + (2 * tile * DT + (w4 >> 1)) * 1024 + 16 * lane;
#pragma unroll
      for (int i = 0; i < SP; i++) {
        *(v8bf*)(w + PS * i * 1024) = bf16x8_of_e4m3(raw[i].x, raw[i].y, sc);
        *(v8bf*)(w + (PS * i + DT) * 1024) = bf16x8_of_e4m3(raw[i].z, raw[i].w, sc);
      }
    }
  };
  auto meet = [&]() {  // LDS reads and writes are done; loads stay in flight
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
  };

  v16f sc[NC][2];
  // weights of 8 tokens: tile, first or second eight of the lane's 16; FINE: and what their rounding left
  v8bf pf[NC][4], pl[FINE ? NC : 1][4];
  auto sees = [&](int u) { return u * kUnit < whi && u * kUnit + kUnit > wlo; };
  auto mul = [](const v8bf& x, const v8bf& y, const v16f& z) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, z, 0, 0, 0);
  };
  // A product phase is a run of stages of four operands, read a stage ahead (two
  // ahead: 3% slower):
  // the scores of step u, then the weighted values of step u - 1.
  constexpr int KST = DS / 2, VST = DT;
  v8bf f[2][4];
  auto read_stage = [&](int st, const uint8_t* kb, const uint8_t* vb) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if (st < KST) f[st & 1][e] = *(const v8bf*)(kb + ((e & 1) * DS + 2 * st + (e >> 1)) * 1024 + 16 * lane);
      else f[st & 1][e] = *(const v8bf*)(vb + (4 * (st - KST) + e) * 1024 + 16 * lane);
    }
  };
  auto multiply_stage = [&](int st) {
#pragma unroll
    for (int e = 0; e < 4; e++)
#pragma unroll
      for (int c = 0; c < NC; c++) {
        if (st < KST) {  // tile e % 2, dims 16 (2 st + e / 2) ..
          sc[c][e & 1] = mul(f[st & 1][e], qf[c][2 * st + (e >> 1)], sc[c][e & 1]);
        } else {         // operand 4 (st - KST) + e: tokens / DT, dims % DT
          const int i = 4 * (st - KST) + e;
          o[c][i % DT] = mul(f[st & 1][e], pf[c][i / DT], o[c][i % DT]);
          if constexpr (FINE) o[c][i % DT] = mul(f[st & 1][e], pl[c][i / DT], o[c][i % DT]);
        }
      }
  };
  auto products = [&](auto from, auto to, const uint8_t* kb, const uint8_t* vb) {
    constexpr int F = decltype(from)::value, E = decltype(to)::value;
    if constexpr (F == 0) {
#pragma unroll
      for (int c = 0; c < NC; c++)
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
          for (int e = 0; e < 16; e++) sc[c][t][e] = 0.f;
    }
    read_stage(F, kb, vb);
#pragma unroll
    for (int st = F; st < E; st++) {
      if (st + 1 < E) read_stage(st + 1, kb, vb);
      __builtin_amdgcn_sched_barrier(0);
      multiply_stage(st);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // rare: step u holds a NaN code among tokens that not every row of the workgroup sees
  auto mark_nans = [&](int u) {
#pragma unroll 1
    for (int t = 0; t < 2; t++) {
      const int T = u * kUnit + 32 * t + 16 * hf;
      int pg = T < head.end(u * kUnit, hi_max) ? head.row(u * kUnit, table)[(T - head.origin(u * kUnit)) >> a.kv.lp] : -1;
      pg = pg >= 0 && pg < a.kv.n_pages ? pg : -1;
      const uint8_t* vc = a.kv.vc + (((int64_t)(pg < 0 ? 0 : pg) * a.kv.H + h) << sh) + ((T - head.origin(u * kUnit)) & (P - 1));
#pragma unroll 1
      for (int d = 0; d < DT; d++) {
        const mx_u4 w = *(const mx_u4*)(vc + (int64_t)(32 * d + n) * P);
        v8bf isn[2];
#pragma unroll
        for (int e = 0; e < 16; e++)
          isn[e >> 3][e & 7] = (__bf16)(pg >= 0 && ((nan_bytes(w[e >> 2]) >> (8 * (e & 3) + 7)) & 1u) ? 1.f : 0.f);
#pragma unroll
        for (int c = 0; c < NC; c++) {
          v8bf vis[2];
#pragma unroll
          for (int e = 0; e < 16; e++)
            vis[e >> 3][e & 7] = (__bf16)(T + e >= vlo[c] && T + e < head.end(u * kUnit, vhi[c]) ? 1.f : 0.f);
          v16f hit;
#pragma unroll
          for (int e = 0; e < 16; e++) hit[e] = 0.f;
          hit = mul(isn[0], vis[0], hit);
          hit = mul(isn[1], vis[1], hit);
#pragma unroll
          for (int e = 0; e < 16; e++) nanned[c] |= hit[e] > 0.f ? uint64_t(1) << (16 * d + e) : 0;
        }
      }
    }
  };
  // weights of step u from its scores
  auto softmax = [&](int u) {
    const int T = u * kUnit;
    bool mask = T + kUnit > whi_all || T < wlo_all || head.gap(u * kUnit);
    int unread = 0;  // tiles whose 16 tokens of the lane cannot be read
    if (bad_at_[u & 3] == u) {
      mask = true;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        const int at = T + 32 * t + 16 * hf;
        const int pg = at < head.end(u * kUnit, hi_max) ? head.row(u * kUnit, table)[(at - head.origin(u * kUnit)) >> a.kv.lp] : -1;
        unread |= pg >= 0 && pg < a.kv.n_pages ? 0 : 1 << t;
      }
    }
#pragma unroll
    for (int c = 0; c < NC; c++) {
      if (mask) {
#pragma unroll
        for (int t = 0; t < 2; t++) {
          const int at = T + 32 * t + 16 * hf;
          const int lo = (unread >> t) & 1 ? 16 : vlo[c] - at, hi = head.end(u * kUnit, vhi[c]) - at;
          const uint32_t up = hi >= 16 ? 0xFFFFu : hi <= 0 ? 0u : (1u << hi) - 1u;
          const uint32_t seen = lo >= 16 ? 0u : lo <= 0 ? up : up & ~((1u << lo) - 1u);
#pragma unroll
          for (int e = 0; e < 16; e++) sc[c][t][e] = (seen >> e) & 1u ? sc[c][t][e] : -INFINITY;
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 32; e++) mx = fmaxf(mx, sc[c][e >> 4][e & 15]);
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
      mx = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])) * scale;
      // The maximum in use may lag by up to 2^8 (weights up to 256 lose no
      // precision), so O is rescaled in few of the steps.
      if (__any(mx > m[c] + 8.f)) {
        const float mn = fmaxf(m[c], mx), mu = mn == -INFINITY ? 0.f : mn;
        const float al = __builtin_amdgcn_exp2f(m[c] - mu);  // first tokens: 2^-inf = 0
        m[c] = mn;
        l[c] *= al;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
          for (int e = 0; e < 16; e++) o[c][d][e] *= al;
      }
      const float mu = m[c] == -INFINITY ? 0.f : m[c];
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 32; e++) {
        const float p = __builtin_amdgcn_exp2f(fmaf(sc[c][e >> 4][e & 15], scale, -mu));  // masked: 2^-inf = 0
        sum[e & 3] += p;
        const __bf16 hi = (__bf16)p;
        pf[c][e >> 3][e & 7] = hi;
        if constexpr (FINE) pl[c][e >> 3][e & 7] = (__bf16)(p - (float)hi);
      }
      l[c] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
  };

  // the phases of attn_prompt
  if (tid < 4) nan_at_[tid] = bad_at_[tid] = -1;
  __syncthreads();
  const int e0 = u0 < u1 ? entry_at(u0) : -1, e1 = u0 + 1 < u1 ? entry_at(u0 + 1) : -1;
  int pg0 = page_of(u0, e0), pg1 = page_of(u0 + 1, e1);
  if (u0 < u1) fetch(u0, pg0);
  // the maximum and the mask's -infinity want a positive scale
  const uint32_t flip = a.scale2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
  for (int c = 0; c < NC; c++)
#pragma unroll
    for (int d = 0; d < DS; d++) {
      mx_u4 w = __builtin_bit_cast(mx_u4, qf[c][d]) ^ flip;
      if (none) w = zero_or_nan(w);
      qf[c][d] = __builtin_bit_cast(v8bf, w);
    }
  if (u0 < u1) stage(u0, pg0);
  meet();
  if (!keys) meet();
  for (int u = u0; u <= u1; u++) {
    const bool more = u + 1 < u1;
    const int e2 = u + 2 < u1 ? entry_at(u + 2) : -1;
    if (more) fetch(u + 1, pg1);
    {
      const bool s_now = u < u1 && sees(u), w_now = u > u0 && sees(u - 1);
      const uint8_t *kb = lds_ + ((u - u0) & 1) * KB, *vb = lds_ + 2 * KB + ((u - u0 + 1) & 1) * VB;
      using First = std::integral_constant<int, 0>;
      using Middle = std::integral_constant<int, KST>;
      using Last = std::integral_constant<int, KST + VST>;
      if (w_now && nan_at_[(u - 1) & 3] == u - 1) mark_nans(u - 1);
      if constexpr (FINE) {
        // Weights first, which then live no longer than scores do: with both terms of them beside the
        // scores 66 registers were spilled (D = 64)
        if (w_now) products(Middle{}, Last{}, kb, vb);
#pragma unroll
        for (int c = 0; c < NC; c++) {
          sc[c][0] = sc[c][1] = v16f{};
#pragma unroll
          for (int e = 0; e < 4; e++) pf[c][e] = pl[c][e] = v8bf{};
        }
        if (s_now) products(First{}, Middle{}, kb, vb);
      } else {
        if (s_now) products(First{}, Middle{}, kb, vb);
        if (w_now) products(Middle{}, Last{}, kb, vb);
      }
    }
    meet();
    if (u < u1 && sees(u)) softmax(u);
    if (more) stage(u + 1, pg1);
    pg1 = page_of(u + 2, e2);
    if (keys || u < u1) meet();
  }
  if (MODE == kHead || parts > 1) {
#pragma unroll
    for (int c = 0; c < NC; c++) {
      l[c] += __shfl_xor(l[c], 32);
      if (rho[c] >= R) continue;
      const uint32_t at = (uint32_t)rho[c] / G;
      float* pp = MODE == kHead
                      ? a.sums + ((part * a.kv.total_q + s.row0 + at) * a.Hq + (int64_t)h * G + (rho[c] - at * G)) * (D + kPartPad)
                      : a.part + ((int64_t)at_.slot * ROWS + (rho[c] - wg0)) * (D + kPartPad);
#pragma unroll
      for (int d = 0; d < DT; d++)
#pragma unroll
        for (int x = 0; x < 4; x++) {
          v4f y;
#pragma unroll
          for (int e = 0; e < 4; e++)
            y[e] = (nanned[c] >> (16 * d + 4 * x + e)) & 1 ? __uint_as_float(0x7FC00000u) : o[c][d][4 * x + e];
          *(v4f*)(pp + 32 * d + 8 * x + 4 * hf) = y;
        }
      if (hf == 0) *(float2*)(pp + D) = make_float2(m[c], l[c]);
    }
    return;
  }
  // through LDS, so that a row's stores lie side by side: a wave's rows are its own
  __syncthreads();
  uint8_t* out = lds_ + wave * (32 * NC * OUT);
#pragma unroll
  for (int c = 0; c < NC; c++) {
    l[c] += __shfl_xor(l[c], 32);
    const float inv = l[c] > 0.f || l[c] != l[c] ? 1.0f / l[c] : 0.f;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int x = 0; x < 4; x++) {  // dims 32 d + 8 x + 4 h .. + 3
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; e++)
          y[e] = (nanned[c] >> (16 * d + 4 * x + e)) & 1 ? __uint_as_float(0x7FC00000u) : o[c][d][4 * x + e] * inv;
        uint2 w;
        w.x = bf16_bits(y[0]) | (bf16_bits(y[1]) << 16);
        w.y = bf16_bits(y[2]) | (bf16_bits(y[3]) << 16);
        *(uint2*)(out + (32 * c + n) * OUT + 64 * d + 16 * x + 8 * hf) = w;
      }
    if (a.lse && hf == 0 && rho[c] < R) {
      const uint32_t at = (uint32_t)rho[c] / G;
      a.lse[(s.row0 + at) * a.Hq + (int64_t)h * G + (rho[c] - at * G)] =
          l[c] == 0.f ? -INFINITY : (m[c] + __builtin_amdgcn_logf(l[c])) * kLn2;
    }
  }
#pragma unroll
  for (int i = 0; i < NC * D / 16; i++) {
    const int row = (i * 64 + lane) / (D / 8), d = 8 * (lane % (D / 8));
    const uint32_t rc = rho0 + row, at = rc / G;
    const mx_u4 w = *(const mx_u4*)(out + row * OUT + 2 * d);
    if (rc < (uint32_t)R) *(mx_u4*)(a.o + (s.row0 + at) * a.o_stride + ((int64_t)h * G + (rc - at * G)) * D + d) = w;
  }
}

// Results of the parts of a tile: O = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k,
// M the largest m_k, in the order of the parts.  One thread for four dims of a
// row, rows of ROWS as the tile's workgroups have them.  Eight parts are read at
// once: the loads' latency bounds it (some 3 us with the launch for 16 parts).
template <int D, int ROWS, int MODE>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  constexpr int T4 = D / 4, AHEAD = 8;
  const uint32_t G = (uint32_t)a.G, H = (uint32_t)a.kv.H, cut = blockIdx.x / H, h = blockIdx.x - cut * H;
  __shared__ int64_t scan_[256 / 64 + 2];
  PromptTile<ROWS, MODE> t;
  if (!t.template find<256>(a, cut + (MODE == kBehind ? a.whole : 0), a.parts, scan_)) return;
  if (t.parts == 1) return;  // its workgroup has written O
  const int parts = t.parts, at = blockIdx.y * 256 + threadIdx.x, r = at / T4, d = at % T4 * 4;
  if (t.wg0 + r >= t.R) return;
  const int64_t step = (int64_t)H * ROWS * (D + kPartPad);  // to the next part
  const float* p = a.part + (((int64_t)cut * a.parts * H + h) * ROWS + r) * (D + kPartPad);
  float M = -INFINITY, L = 0.f;
  v4f o = v4f{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < parts; k += AHEAD) {
    v4f po[AHEAD];
    float2 ml[AHEAD];
#pragma unroll
    for (int e = 0; e < AHEAD; e++) {
      const float* q = p + min(k + e, parts - 1) * step;
      po[e] = *(const v4f*)(q + d);
      ml[e] = *(const float2*)(q + D);
    }
    float mx = M;
#pragma unroll
    for (int e = 0; e < AHEAD; e++) mx = fmaxf(mx, ml[e].x);
    const float mu = mx == -INFINITY ? 0.f : mx, al = __builtin_amdgcn_exp2f(M - mu);
    M = mx;
    L *= al;
#pragma unroll
    for (int c = 0; c < 4; c++) o[c] *= al;
#pragma unroll
    for (int e = 0; e < AHEAD; e++) {
      if (k + e >= parts) break;
      const float w = __builtin_amdgcn_exp2f(ml[e].x - mu);
      L += w * ml[e].y;
#pragma unroll
      for (int c = 0; c < 4; c++) o[c] += w * po[e][c];
    }
  }
  const uint32_t rc = t.wg0 + r, tok = rc / G;
  const int64_t row = t.s.row0 + tok, hd = (int64_t)h * G + (rc - tok * G);
  const float inv = L > 0.f || L != L ? 1.0f / L : 0.f;
  uint2 w;
  w.x = bf16_bits(o[0] * inv) | (bf16_bits(o[1] * inv) << 16);
  w.y = bf16_bits(o[2] * inv) | (bf16_bits(o[3] * inv) << 16);
  *(uint2*)(a.o + row * a.o_stride + hd * D + d) = w;
  if (a.lse && d == 0) a.lse[row * a.Hq + hd] = L == 0.f ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

struct Plan {
  int nc;             // column tiles of a decode tile; 0: attn_prompt
  int rows;           // of a prompt tile
  int parts;          // of its steps
  int64_t blocks;
};

// Few rows or many.  A wave of attn_decode has 16 rows (32 for D = 64, in twice
// the registers) and every tile reads the cache again; attn_prompt reads it once
// for all rows, but widens it for 128 or 256 of them and joins its parts by
// another launch.  So the choice goes by the rows of a head and the steps of all
// heads.  us in a graph over two caches in turn, attn_decode / attn_prompt, 32 heads over 8 (D = 256: 24 over 4):
//   D = 64   4 rows, 1 x 1024 9.3 / 10.9; 16 rows 10.8 / 11.5, 1 x 4096 14.6 / 15.1
//            20 rows, 1 x 4096 18.1 / 15.1, 16 x 2048 21.2 / 21.1
//            40 rows, 1 x 4096 20.3 / 15.3, 64 x 2048 61 / 56, 1 x 32768 29 / 41
//            80 rows, 16 x 2048 36 / 29
//   D = 128  8 rows, 1 x 1024 12.1 / 12.4, 1 x 4096 15.7 / 16.8, 8 x 1000 13.8 / 15.0
//            16 rows, 1 x 1024 14.2 / 12.6, 1 x 8192 21.9 / 21.2, 16 x 2048 25.0 / 25.8
//            20 rows, 1 x 4096 20 / 17, 64 x 2048 88 / 66, 1 x 131071 83 / 83
//            40 rows, 1 x 32768 43 / 47, 64 x 2048 124 / 74
//   D = 256  6 rows, 1 x 1024 15.5 / 14.6, 8 x 1024 17.3 / 16.2, 32 x 1024 23 / 29, 1 x 16384 23 / 33
//            18 rows, 1 x 1024 21 / 15, 64 x 2048 97 / 69
bool many_rows(const KvArgs& kv, int64_t R) {
  constexpr int64_t kAny = INT64_MAX;
  int64_t most;  // steps up to which attn_prompt is the faster one
  if (kv.D == 64) most = R <= 16 ? 0 : R <= 64 ? 2048 : kAny;
  else if (kv.D == 128) most = R <= 8 ? 0 : R <= 16 ? 1024 : kAny;
  else most = R <= 16 ? 512 : kAny;
  return kv.n_seqs * kv.H * cdiv(kv.max_kv, kUnit) <= most;
}
// Rows of a workgroup, and workgroups that the chip holds at once.  D = 128: 256
// rows, 128 where no sequence has more (two workgroups a compute unit, fewer idle
// waves; 2 x 4096 in 4096, 40 heads over 8, 411 us with 128 rows and 376 with 256,
// 16 x 64 in 1024 50 and 42, 16 x 5 in 2048, 32 heads, 26 and 35).
int prompt_rows(int D, int64_t R) { return D == 128 && R > 128 ? 256 : 128; }
int prompt_slots(int D, int64_t R) { return D == 64 ? 768 : D == 128 && R <= 128 ? 512 : 256; }

// window: 0 where rows see everything before them or more
Plan plan_attention(const KvArgs& kv, int64_t G, int64_t window) {
  Plan p;
  const int64_t R = kv.max_q * G, rows = prompt_rows(kv.D, R), slots = prompt_slots(kv.D, R);
  p.rows = (int)rows;
  p.parts = 1;
  if (many_rows(kv, R)) {
    p.nc = 0;
    p.blocks = std::min<int64_t>(kv.n_seqs * kv.H * cdiv(R, rows), kv.H * (kv.total_q * G / rows + kv.n_seqs));
    // at most as parts_of has them
    const int64_t most = window > 0 ? std::min<int64_t>(kv.max_kv, window + rows / G + 2) : kv.max_kv;
    const int64_t best = (int64_t)(2.0 * sqrt((double)cdiv(most, kUnit)));
    p.parts = (int)std::max<int64_t>(std::min(slots / p.blocks, best), 1);
    return p;
  }
  p.nc = R > 16 && kv.D == 64 ? 2 : 1;  // wider heads: the registers of 16 rows
  p.blocks = kv.D == 256 ? kMaxShares / 2 : kMaxShares;  // what the chip holds at once
  return p;
}

template <int MODE, bool FINE = false>
void launch_prompt(int rows, unsigned blocks, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(blocks);
  if (a.kv.D == 64) hipLaunchKernelGGL((attn_prompt32<64, 1, 4, 3, MODE, FINE>), grid, dim3(256), 0, s, a);
  else if (a.kv.D == 256) hipLaunchKernelGGL((attn_prompt<256, 1, 8, MODE, FINE>), grid, dim3(512), 0, s, a);
  else if (rows == 128) hipLaunchKernelGGL((attn_prompt32<128, 1, 4, 2, MODE, FINE>), grid, dim3(256), 0, s, a);
  else if constexpr (MODE != kBehind || !FINE)  // of sequences with few rows the tiles have 128
    hipLaunchKernelGGL((attn_prompt32<128, 1, 8, 2, MODE, FINE>), grid, dim3(512), 0, s, a);
}
// tiles: of all heads
template <int MODE>
void launch_join(int rows, int64_t tiles, const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)tiles, (unsigned)(rows * a.kv.D / 4 / 256));
  if (a.kv.D == 64) hipLaunchKernelGGL((attn_join<64, 128, MODE>), grid, dim3(256), 0, s, a);
  else if (a.kv.D == 128 && rows == 128) hipLaunchKernelGGL((attn_join<128, 128, MODE>), grid, dim3(256), 0, s, a);
  else if (a.kv.D == 128) hipLaunchKernelGGL((attn_join<128, 256, MODE>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((attn_join<256, 128, MODE>), grid, dim3(256), 0, s, a);
}
template <int MODE>
void launch_decode(int nc, unsigned blocks, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(blocks), block(64 * kDecWaves);
  if (a.kv.D == 64 && nc == 1) hipLaunchKernelGGL((attn_decode<64, 1, MODE>), grid, block, 0, s, a);
  else if (a.kv.D == 64) hipLaunchKernelGGL((attn_decode<64, 2, MODE>), grid, block, 0, s, a);
  else if (a.kv.D == 128) hipLaunchKernelGGL((attn_decode<128, 1, MODE>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attn_decode<256, 1, MODE>), grid, block, 0, s, a);
}

// bound on the tiles of all heads
int64_t tiles_of(const KvArgs& kv, int64_t G, int64_t rows, int64_t max_q) {
  return std::min<int64_t>(kv.n_seqs * kv.H * cdiv(max_q * G, rows), kv.H * (kv.total_q * G / rows + kv.n_seqs));
}
int64_t tiles_of(const KvArgs& kv, int64_t G, int64_t rows) { return tiles_of(kv, G, rows, kv.max_q); }
int best_parts(int64_t steps) { return (int)std::max<int64_t>((int64_t)(2.0 * sqrt((double)steps)), 1); }

// us of a prompt workgroup over some steps, `wgs` of them at work at once, `fill` of
// its rows used
double wg_time(int D, int64_t rows, double fill, int64_t wgs, double steps) {
  const bool crowded = wgs > 256;
  const double step = D == 64     ? (crowded ? 1.4 + 0.8 * fill : 1.3 + 0.2 * fill)
                      : D == 256  ? 1.6 + 1.1 * fill
                      : rows == 256 ? 1.4 + 0.45 * fill
                      : crowded   ? 1.5 + 0.9 * fill
                                  : 1.4 + 0.2 * fill;
  return step * steps + (D == 256 ? 10. : 6.);
}
// tiles (of at most `most`, for which there is to be room) cut into the parts that take
// the least time; `sums`: us to write and read one part of each, `join`: us that
// joining takes beside that
double cut_time(int D, int64_t rows, double fill, int64_t tiles, int64_t most, int64_t steps, double sums, double join, int* parts) {
  double least = 1e30;
  const int64_t slots = prompt_slots(D, rows);
  for (int64_t k = 1; k <= best_parts(steps) && (k == 1 || most * k <= 4 * slots); k++) {
    const double t = (double)cdiv(tiles * k, slots) * wg_time(D, rows, fill, std::min(tiles * k, slots), (double)steps / (double)k) +
                     (k > 1 || join == 0. ? sums * (double)k + join : 0.);
    if (t < least) {
      least = t;
      *parts = (int)k;
    }
  }
  return least;
}
// us of attn_decode over the groups' rows, in equal shares of all blocks
double decode_time(int D, int64_t rows, int64_t tiles, int64_t blocks) {
  const double shares = D == 256 ? kMaxShares / 2 : kMaxShares, x = (double)(tiles * blocks) / shares;
  const double parts = std::min(shares / (double)tiles, (double)blocks);  // of a tile, to be joined
  const double join = parts > 1. ? 0.08 * (double)std::min<int64_t>(rows, D == 64 ? 32 : 16) * sqrt(parts) : 0.;
  const double work = D == 256 ? 18. + 3.3 * x : D == 128 ? 13. + 3. * x : rows > 16 ? 18. + 2.8 * x : 11. + 1.9 * x;
  return work + join;
}
// us of joining the pieces of a tile
double join_time(int D, int64_t rows, int64_t pieces) {
  const double each = D == 64 ? 0.05 : D == 128 ? 0.13 : 0.25;
  return pieces > 1 ? 1.4 + each * (double)std::min<int64_t>(rows, D == 64 ? 32 : 16) * sqrt((double)pieces) : 0.;
}
// us of attn_decode over sequences and their prefixes, `pieces` a tile (0: equal shares of all blocks)
double few_time_of(int D, int64_t rows, int64_t tiles, int64_t blocks, int64_t pieces) {
  const double shares = D == 256 ? kMaxShares / 2 : kMaxShares, t = (double)tiles / shares, x = t * (double)blocks;
  if (pieces == 0) {
    if (D == 64) return rows > 16 ? 22.5 + 1.9 * x + 3. * t : 12.9 + 1.6 * x + 4.2 * t;
    return D == 128 ? 15.3 + 2.7 * x + 4.3 * t : 11.8 + 3.1 * x + 8.4 * t;
  }
  const double join = join_time(D, rows, pieces);
  if (D == 64) return (rows > 16 ? 12.5 + 2.6 * x : 9.6 + 2.3 * x) + join;
  return (D == 128 ? 10.8 + 3.2 * x : 12.5 + 0.6 * x + 3.4 * (double)cdiv(blocks, pieces)) + join;
}
// us of the sequences' launch behind the groups', beside what it takes for a block of each: `t` times the tiles
// and pieces that the chip holds
double tail_time(int D, int64_t rows, int64_t tiles, int64_t blocks, int64_t pieces) {
  const double t = (double)(tiles * pieces) / (D == 256 ? kMaxShares / 2 : kMaxShares), full = std::max(t, 1.);
  const double each = (double)cdiv(blocks, pieces);
  const double time = D == 64 ? 2.5 * t + 2.1 * full * each + 4. * (full - 1.) : D == 128 ? 6. * t + 4. * full * each
                                                                                         : 6. * t + 3.3 * full * each + 5. * (full - 1.);
  return time + join_time(D, rows, pieces);
}

// The three ways by their expected times, whose numbers are fitted to 450 random calls (1 to 8 groups of 2 to 64
// sequences, 1 to 700 new tokens, prefixes of 10 to 60000; outside of that they are extrapolation); 450 others took
// 1.1% longer than with always the best of the three.  us, measured, single tokens of 32 heads over 8 behind one prefix
// (D = 256: 24 over 4), 100 own tokens, in one attn_decode / in two launches:
//   D = 64   8 sequences behind 8000 18 / 25, 16 26 / 27, 32 40 / 32, 8 behind 32000 40 / 37
//   D = 128  4 behind 1000 12 / 20, 8 behind 8000 25 / 32, 16 37 / 34, 32 60 / 39, 8 behind 32000 59 / 46
//   D = 256  8 behind 8000 31 / 40, 16 44 / 49, 32 69 / 52, 8 behind 32000 69 / 56
// and more rows of each of 32 sequences behind 16000 / 2000, D = 128, in one prompt launch / in two:
//   32 rows 281 / 119 and 54 / 47, 64 rows 328 / 210 and 80 / 63, 128 rows 330 / 294 and 73 / 89.
// attn_decode over sequences and prefixes in pieces rather than equal shares where there are no more than 8 blocks a
// workgroup (of the 450 calls those with 2 to 4 took 0.72 to 0.87 of the time, with 4 to 8 0.9, with more 1.0 to 1.25,
// as sequences differ in length).
constexpr int64_t kMostBlocks = 1 << 22;  // of a launch
constexpr int64_t kNoTile = 8;            // rows of a sequence and key head that do not take a prompt tile of their own
constexpr int64_t kSpaced = 256;          // rows of a sequence and key head, with those before the next, that groups take
constexpr int64_t kFineRows = 64;         // of a sequence and key head: eight tokens of eight heads
PrefixPlan plan_prefix_of(const AttnArgs& a) {
  const KvArgs &kv = a.kv, &prefix = a.prefix;
  const int D = kv.D;
  const int64_t Rs = kv.max_q * a.G, Rg = a.group_q * a.G, row_bytes = (D + kPartPad) * 4;
  const int64_t head_steps = cdiv(prefix.max_kv, kUnit), own_steps = cdiv(kv.max_kv, kUnit), steps = head_steps + own_steps;
  constexpr double kRate = 4.8e6;  // bytes a us
  auto decode_nc = [&](int64_t R) { return R > 16 && D == 64 ? 2 : 1; };
  auto decode_part = [&](int nc) { return (size_t)4 * kMaxShares * 16 * nc * (D + 2) * 4; };
  const int64_t shares = D == 256 ? kMaxShares / 2 : kMaxShares;

  // tiles of the sequences' rows, all steps
  PrefixPlan one = {};
  one.behind = true;
  one.fine = Rs <= kFineRows;
  one.rows = prompt_rows(D, Rs);
  const int64_t slots = prompt_slots(D, Rs), most = tiles_of(kv, a.G, one.rows);
  // tiles to be expected: each sequence's last one half full, but one of each
  const int64_t tiles =
      std::min(most, kv.H * std::max(kv.n_seqs, kv.total_q * a.G / one.rows + (kv.n_seqs + 1) / 2));
  one.whole = (int)(tiles / slots * slots / kv.H);
  const int64_t rest = tiles - one.whole * kv.H;  // behind the last full round
  one.parts = 1;
  const double one_fill = (double)std::min<int64_t>(Rs, one.rows) / (double)one.rows;
  double one_time = (double)(one.whole * kv.H) / (double)slots * wg_time(D, one.rows, one_fill, slots, (double)steps);
  if (rest)
    one_time += cut_time(D, one.rows, one_fill, rest, most - one.whole * kv.H, steps,
                         one_fill * (double)(rest * one.rows * row_bytes) * 2. / kRate, 4. + 0.03 * (double)rest, &one.parts);
  if (one.parts == 1) one.whole = (int)(most / kv.H);
  one.cut = most - one.whole * kv.H;
  one.blocks = one.whole * kv.H + one.cut * one.parts;
  one.part = (size_t)(one.cut * one.parts * one.rows * row_bytes);
  one_time = 0.92 * one_time + (D == 64 ? 3.7 : D == 256 ? 1.9 : one.rows == 128 ? 4.9 : 10.3);
  if (one.fine && D == 128) one_time *= 1.15;  // the second terms; with other heads the times' spread is larger
  if (Rs <= kNoTile) one_time = 1e30;  // tiles filled to a sixteenth: of 252 such calls none took less than 0.98 of the others' time

  // the same in attn_decode
  const int nc = decode_nc(Rs);
  const int64_t few_tiles = tiles_of(kv, a.G, 16 * nc), few_blocks = cdiv(steps, kDecWaves);
  const bool in_pieces = few_tiles <= shares && few_tiles * few_blocks <= 8 * shares;
  const int64_t few_pieces = in_pieces ? std::min(shares / few_tiles, few_blocks) : 0;
  const double few_time = few_time_of(D, Rs, few_tiles, few_blocks, few_pieces);

  // groups, then sequences
  PrefixPlan two = {};
  two.fine = Rs <= kFineRows;
  two.parts = 1;
  two.tail_nc = nc;
  // as many pieces of a tile as fill the chip
  two.pieces = (int)std::max<int64_t>(std::min(shares / few_tiles, cdiv(kv.max_kv, kBlock)), 1);
  two.tail_blocks = few_tiles * two.pieces;
  if (two.pieces > 1) two.part = decode_part(nc);
  double two_time = D == 256 ? 10.7 : 8.4;
  two_time += tail_time(D, Rs, few_tiles, cdiv(own_steps, kDecWaves), two.pieces);
  if (many_rows(prefix, Rg)) {
    // 256 rows a tile where that is not a fifth more of them than in tiles of 128
    two.rows = prompt_rows(D, cdiv(Rg, 256) * 256 * 5 < cdiv(Rg, 128) * 128 * 6 ? Rg : 128);
    const int64_t group_tiles = tiles_of(prefix, a.G, two.rows, a.group_q), room = tiles_of(prefix, a.G, two.rows);
    two_time += cut_time(D, two.rows, (double)std::min<int64_t>(Rg, two.rows) / (double)two.rows, group_tiles, room, head_steps,
                         (double)(kv.total_q * a.Hq * row_bytes) * 2. / kRate, 0., &two.parts);
    two.blocks = room * two.parts;
  } else {
    two.nc = decode_nc(Rg);
    two.blocks = shares;
    two.part = std::max(two.part, decode_part(two.nc));
    two_time += decode_time(D, Rg, tiles_of(prefix, a.G, 16 * two.nc, a.group_q), cdiv(head_steps, kDecWaves));
  }
  two.sums = (size_t)(two.parts * kv.total_q * a.Hq * row_bytes);

  // sequences of more than 256 rows fill their tiles without a group, and need no sums; rows
  // between them would be the groups' work too
  const int64_t spaced = std::max(kv.max_q, kv.total_q / kv.n_seqs) * a.G;
  if (spaced > kSpaced || two.blocks > kMostBlocks || two.tail_blocks > kMostBlocks) two_time = 1e30;
  if (few_time <= std::min(one_time, two_time)) {
    PrefixPlan few = {};
    few.behind = true;
    few.nc = nc;
    few.parts = 1;
    few.pieces = (int)few_pieces;
    few.blocks = in_pieces ? cdiv(few_tiles * few_pieces, 8) * 8 : shares;
    few.part = decode_part(nc);
    return few;
  }
  return one_time <= two_time ? one : two;
}

}  // namespace

int64_t attention_blocks(const KvArgs& kv, int64_t G) { return plan_attention(kv, G, 0).blocks; }

size_t attention_workspace_bytes(const KvArgs& kv, int64_t G) {
  const Plan p = plan_attention(kv, G, 0);  // a window takes no more
  if (p.nc > 0) return (size_t)kCounterBytes + (size_t)4 * kMaxShares * 16 * p.nc * (kv.D + 2) * 4;
  if (p.parts == 1) return 0;
  return (size_t)kCounterBytes + (size_t)(p.blocks * p.parts * p.rows) * (kv.D + kPartPad) * 4;
}

hipError_t launch_attention(AttnArgs a, void* ws, hipStream_t s) {
  const Plan p = plan_attention(a.kv, a.G, a.causal ? a.window : 0);
  a.cnt = (uint32_t*)ws + 16;
  a.part = (float*)((uint8_t*)ws + kCounterBytes);
  a.parts = p.parts;
  if (p.nc > 0) {
    launch_decode<kPlain>(p.nc, (unsigned)p.blocks, a, s);
  } else {
    launch_prompt<kPlain>(p.rows, (unsigned)(p.blocks * p.parts), a, s);
    if (p.parts > 1) launch_join<kPlain>(p.rows, p.blocks, a, s);
  }
  return hipGetLastError();
}

PrefixPlan plan_prefix(const AttnArgs& a) { return plan_prefix_of(a); }

// For every plan within the bounds of `a`, which does not fall as any of them rises: plans do not grow with their
// calls, as a smaller call may be cut into more parts.
size_t attention_prefix_workspace_bytes(const AttnArgs& a) {
  const KvArgs& kv = a.kv;
  const int D = kv.D;
  const int64_t row_bytes = (D + kPartPad) * 4;
  const int64_t total = std::min(kv.total_q, kv.n_seqs * (kSpaced / a.G + 1)) * a.Hq;  // rows that may have sums
  // Tiles in parts, of 128 rows or for D = 128 of 256, are at most four times those that the chip holds, and
  // a tile has at most best_parts of them.
  const int64_t rows = D == 128 ? 256 : 128, most = 4 * prompt_slots(D, rows) * rows;
  const int64_t head_steps = cdiv(a.prefix.max_kv, kUnit), steps = head_steps + cdiv(kv.max_kv, kUnit);
  const int64_t decode = (int64_t)4 * kMaxShares * 16 * (D == 64 ? 2 : 1) * (D + 2) * 4;
  const int64_t sums = std::max(total, std::min(best_parts(head_steps) * total, most)) * row_bytes;
  const int64_t tiles = tiles_of(kv, a.G, rows) * rows;
  const int64_t own = kv.max_q * a.G > kNoTile ? std::min(best_parts(steps) * tiles, most) * row_bytes : 0;
  return (size_t)(kCounterBytes + std::max(sums + decode, own));
}

hipError_t launch_attention_prefix(AttnArgs a, const PrefixPlan& p, void* ws, hipStream_t s) {
  uint8_t* at = (uint8_t*)ws + kCounterBytes;
  a.cnt = (uint32_t*)ws + 16;
  a.sums = (float*)at;
  a.part = (float*)(at + p.sums);
  a.parts = a.sums_parts = p.parts;
  a.whole = p.whole;
  a.pieces = p.pieces;
  if (p.behind) {
    if (p.nc > 0) {
      launch_decode<kBehind>(p.nc, (unsigned)p.blocks, a, s);
    } else {
      if (p.fine) launch_prompt<kBehind, true>(p.rows, (unsigned)p.blocks, a, s);
      else launch_prompt<kBehind>(p.rows, (unsigned)p.blocks, a, s);
      if (p.parts > 1) launch_join<kBehind>(p.rows, p.cut, a, s);
    }
    return hipGetLastError();
  }
  AttnArgs head = a;
  head.kv = a.prefix;
  head.causal = 0;
  if (p.nc > 0) launch_decode<kHead>(p.nc, (unsigned)p.blocks, head, s);
  else if (p.fine) launch_prompt<kHead, true>(p.rows, (unsigned)p.blocks, head, s);
  else launch_prompt<kHead>(p.rows, (unsigned)p.blocks, head, s);
  launch_decode<kTail>(p.tail_nc, (unsigned)p.tail_blocks, a, s);
  return hipGetLastError();
}

}  // namespace lowbit
