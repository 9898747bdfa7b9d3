// Pages of the 8-bit cache: the next batch's tables, lengths and reference
// counts from this one's (kv8_fork), and pages in use moved together
// (kv8_compact).
//
// Everything that decides is whole numbers, and every choice goes by the order
// of children and pages, so results do not depend on the order of atomics.
// Pages are chosen by one small kernel (fork) or by chunks of 4096 pages
// (compact); their bytes are moved by a launch that fills the chip, a page's keys
// or values being one run of heads * tokens * dims bytes.
// In a graph, 64 sequences of 33 pages forked 11 us (plan 8.7 alone, rows and copies 4.4 alone; 47
// with 32 layers, whose copies are 33 MB), 200 of 2048 pages 14; 700 pages compacted 7.3 us, 6000 of
// 128 KiB with some 1000 moves 66 (plan 7.3; moves 46, 132 MB read and written, 5.8 TB/s).  Pools of
// more than kNearPages are planned by the same one workgroup over counts in memory: 40 prompts of 8
// beams, 30000 tokens in pages of 16 (600000 entries, 78100 pages) 626 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv8.hpp"

namespace lowbit {
namespace {

constexpr int kPlan = 1024;          // threads of the planning workgroup
constexpr int kPiece = 16384;        // bytes that a workgroup moves at a time
constexpr int kMoveThreads = 256;
constexpr int kRows = 1024;          // table entries written by a workgroup at a time

__device__ __forceinline__ int load_dev(const int* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_dev(int* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void add_dev(int* p, int v) {
  __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// the workgroup's stores and atomics to memory are done
__device__ __forceinline__ void meet() {
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

// sum of the values before this thread's, and of all of them
template <int THREADS>
__device__ __forceinline__ int scan_before(int v, int* lds, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(sum, d);
    sum += lane >= d ? x : 0;
  }
  __syncthreads();  // lds may still be read from the scan before
  if (lane == 63) lds[wave] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; w++) {
    before += w < wave ? lds[w] : 0;
    all += lds[w];
  }
  *total = all;
  return before + sum - v;
}

__host__ __device__ __forceinline__ int64_t pages_of(int64_t tokens, int lp) { return (tokens + (int64_t(1) << lp) - 1) >> lp; }

// What child i takes over and gets.
struct Child {
  int64_t parent;  // -1: none
  int64_t had;     // pages taken over
  int64_t need;    // with the tokens to come
  int64_t len;     // with them
  bool cut;        // fewer tokens than the parent's and those to come
  int64_t tail;    // partly filled page that will be written to, -1: none
};
__device__ __forceinline__ int64_t parent_of(const ForkArgs& a, int64_t i) {
  const int64_t p = a.parents[i];
  return p >= 0 && p < a.n_seqs ? p : -1;
}
// tokens that `width` pages hold, and lengths can count
__device__ __forceinline__ int64_t most_tokens(int64_t width, int lp) { return min(width << lp, int64_t(1) << 30); }
__device__ __forceinline__ int64_t length_of(const ForkArgs& a, int64_t b) {
  const int64_t n = a.lens[b], most = most_tokens(a.width, a.lp);
  return n < 0 ? 0 : n < most ? n : most;
}
__device__ __forceinline__ Child child_of(const ForkArgs& a, int64_t i) {
  Child c;
  c.parent = parent_of(a, i);
  const int64_t most = most_tokens(a.new_width, a.lp);
  const int64_t all = c.parent < 0 ? 0 : length_of(a, c.parent), n = min(all, most);
  int64_t grow = a.grow ? (int64_t)a.grow[i] : a.max_grow;
  grow = grow < 0 ? 0 : grow < a.max_grow ? grow : a.max_grow;
  c.len = min(n + grow, most);
  c.cut = all + grow > c.len;
  c.had = pages_of(n, a.lp);
  c.need = pages_of(c.len, a.lp);
  c.tail = -1;
  if (c.len > n && (n & ((int64_t(1) << a.lp) - 1))) {
    const int64_t p = a.table[c.parent * a.width + c.had - 1];
    if (p >= 0 && p < a.n_pages) c.tail = p;
  }
  return c;
}

__global__ void copy_refs(const int32_t* __restrict__ from, int32_t* __restrict__ to, int64_t n) {
  const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (i < n) to[i] = from[i];
}

constexpr int kLayers = 32;  // given to a launch
struct Layers {
  PageLayer at[kLayers];
  int n;
};
// A table of layers in the workspace: an array among a kernel's arguments that is
// indexed by a variable would be copied to every lane's private memory (1.5 KB; the
// moves below took 4 times as long).
__device__ __forceinline__ void put_layers(PageLayer* to, const Layers& l) {
#pragma unroll
  for (int i = 0; i < kLayers; i++)
    if (i < l.n) to[i] = l.at[i];
}
__global__ void more_layers(PageLayer* to, Layers l) { put_layers(to, l); }

// One workgroup: children of each parent, counts of holders, which tail pages
// are copied, free pages.  Bound by the latency of its steps, each of which needs
// what the one before counted, so the counts lie in LDS where they fit (NEAR).
//
// A tail page of r holders, w of which will write to it: with r > w all of them
// copy and r - w holders stay; with r = w the first one keeps it.  So the writers
// take themselves off its count, and where that leaves 0, the smallest of them is
// written in its place.
constexpr int kNearSeqs = 4096;       // sequences whose children and lengths lie in LDS
// Pages whose counts do: with the sequences' 32 KiB 147 KB of a compute unit's 160; whole turns of
// the workgroup's free pages (4 to a thread).
constexpr int kNearPages = 28672;
constexpr int kFirst = INT32_MIN;     // + child: it keeps the page

template <bool NEAR>
__global__ __launch_bounds__(kPlan) void fork_plan(ForkArgs a, Layers l) {
  __shared__ int lds[kPlan / 64];
  __shared__ int near_children[kNearSeqs], near_lens[kNearSeqs];
  __shared__ __attribute__((aligned(16))) int near_refs[NEAR ? kNearPages : 4];
  const int tid = threadIdx.x;
  const bool near = a.n_seqs <= kNearSeqs;
  auto add = [&](int64_t p, int d) {
    if constexpr (NEAR) atomicAdd(near_refs + p, d);
    else add_dev(a.new_refs + p, d);
  };
  auto count = [&](int64_t p) -> int {
    if constexpr (NEAR) return near_refs[p];
    else return load_dev(a.new_refs + p);
  };
  auto put = [&](int64_t p, int v) {
    if constexpr (NEAR) near_refs[p] = v;
    else store_dev(a.new_refs + p, v);
  };
  auto step = [&]() {
    if constexpr (NEAR) __syncthreads();
    else meet();
  };
  if constexpr (NEAR) {
    constexpr int kRun = 8;
    for (int p0 = 0; p0 < a.n_pages; p0 += kPlan * kRun) {
      int r[kRun];
#pragma unroll
      for (int e = 0; e < kRun; e++) {
        const int p = p0 + e * kPlan + tid;
        r[e] = p < a.n_pages ? a.refs[p] : 0;
      }
#pragma unroll
      for (int e = 0; e < kRun; e++) {
        const int p = p0 + e * kPlan + tid;
        if (p < a.n_pages) near_refs[p] = r[e];
      }
    }
  }
  for (int64_t b = tid; b < a.n_seqs; b += kPlan) {
    if (near) {
      near_children[b] = 0;
      near_lens[b] = (int)length_of(a, b);
    } else {
      store_dev(a.children + b, 0);
    }
  }
  // the first children's, which every step wants, stay in registers
  Child mine = {};
  mine.parent = mine.tail = -1;
  if (tid < a.n_new) mine = child_of(a, tid);
  auto child = [&](int64_t i) { return i < kPlan ? mine : child_of(a, i); };
  if (tid == 0) put_layers(a.layers, l);
  if (near) __syncthreads();
  else meet();
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const int64_t b = i < kPlan ? mine.parent : parent_of(a, i);
    if (b < 0) continue;
    if (near) atomicAdd(near_children + b, 1);
    else add_dev(a.children + b, 1);
  }
  if (near) __syncthreads();
  else meet();
  // A page loses its old holders and gains their children: nothing changes for a
  // sequence that goes on as one.  Teams of threads have a sequence each, four
  // entries of a thread on their way at once.
  constexpr int kAhead = 4;
  int team = 16;
  while (team < kPlan && team * kAhead < a.width) team *= 2;
  for (int64_t b = tid / team; b < a.n_seqs; b += kPlan / team) {
    const int64_t held = pages_of(near ? near_lens[b] : length_of(a, b), a.lp);
    const int children = near ? near_children[b] : load_dev(a.children + b);
    if (children == 1 && held <= a.new_width) continue;
    for (int64_t j0 = tid & (team - 1); j0 < held; j0 += team * kAhead) {
      int p[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; e++) p[e] = j0 + e * team < held ? a.table[b * a.width + j0 + e * team] : -1;
#pragma unroll
      for (int e = 0; e < kAhead; e++) {
        const int d = (j0 + e * team < a.new_width ? children : 0) - 1;
        if (d != 0 && p[e] >= 0 && p[e] < a.n_pages) add(p[e], d);
      }
    }
  }
  step();
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const int64_t t = child(i).tail;
    if (t >= 0) add(t, -1);
  }
  step();
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const int64_t t = child(i).tail;
    if (t < 0) continue;
    // 0 until the first child of such a page comes, less from then on
    if constexpr (NEAR) {
      if (near_refs[t] <= 0) atomicMin(near_refs + t, kFirst + (int)i);
    } else {
      if (load_dev(a.new_refs + t) <= 0)
        __hip_atomic_fetch_min(a.new_refs + t, kFirst + (int)i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
  }
  step();
  // pages that the children need, in their order
  int64_t total = 0;
  int copies = 0, cut = 0;
  for (int64_t i0 = 0; i0 < a.n_new; i0 += kPlan) {
    const int64_t i = i0 + tid;
    int need = 0, copy = 0;
    Child c;
    if (i < a.n_new) {
      c = child(i);
      copy = c.tail >= 0 && count(c.tail) != kFirst + (int)i;
      need = copy + (int)(c.need - c.had);
    }
    int all, all_copies;
    const int before = scan_before<kPlan>(need, lds, &all);
    const int nth = scan_before<kPlan>(copy, lds, &all_copies);
    if (i < a.n_new) {
      a.start[i] = (total + before) * 2 + copy;
      if (copy) {
        a.src[copies + nth] = (int)c.tail;
        a.dst[copies + nth] = (int)(total + before);  // the place of its page among the free ones
      }
      a.new_lens[i] = (int32_t)c.len;
      cut += c.cut;
    }
    total += all;
    copies += all_copies;
  }
  step();
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const int64_t t = child(i).tail;
    if (t >= 0 && count(t) == kFirst + (int)i) put(t, 1);
  }
  step();
  // the first `total` free pages; counts in memory by wide loads, past what L1 may hold of them
  int64_t found = 0;
  constexpr int kRun = NEAR ? 4 : 16;
  if constexpr (!NEAR) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  for (int64_t p0 = 0; p0 < a.n_pages && found < total; p0 += kPlan * kRun) {
    const int64_t p = p0 + tid * kRun;
    const int* counts = NEAR ? near_refs : a.new_refs;
    uint32_t free = 0;
    if (p + kRun <= a.n_pages) {
      mx_u4 r[kRun / 4];
#pragma unroll
      for (int e = 0; e < kRun / 4; e++) r[e] = *(const mx_u4*)(counts + p + 4 * e);
#pragma unroll
      for (int e = 0; e < kRun; e++) free |= r[e / 4][e % 4] == 0 ? 1u << e : 0u;
    } else {
      for (int e = 0; p + e < a.n_pages; e++) free |= counts[p + e] == 0 ? 1u << e : 0u;
    }
    int all;
    int64_t at = found + scan_before<kPlan>(__builtin_popcount(free), lds, &all);
    for (; free && at < total; free &= free - 1, at++) {
      const int64_t page = p + __builtin_ctz(free);
      a.fresh[at] = (int)page;
      put(page, 1);
    }
    found += all;
  }
  if constexpr (NEAR) {
    __syncthreads();
    for (int p = tid; p < a.n_pages; p += kPlan) a.new_refs[p] = near_refs[p];
  }
  if (a.cut) {
    int all;
    (void)scan_before<kPlan>(cut, lds, &all);
    if (tid == 0) *a.cut = all;
  }
  if (tid == 0) {
    *a.n_copies = found >= total ? copies : 0;
    *a.found = min(found, total);
    *a.failed = (int32_t)min(total - min(found, total), (int64_t)INT32_MAX);
  }
}

// piece `piece` of the pages of all layers, page src to page dst
__device__ __forceinline__ void move_piece(const PageLayer* layers, int pieces, int piece, int64_t src, int64_t dst) {
  const int i = piece / pieces;  // `pieces` of the largest layer
  piece -= i * pieces;
  const PageLayer at = layers[i];
  const int half = (int)((at.bytes + kPiece - 1) / kPiece);
  if (piece >= 2 * half) return;
  const bool keys = piece < half;
  const int64_t off = (int64_t)(keys ? piece : piece - half) * kPiece;
  uint8_t* base = keys ? at.k : at.v;
  const uint8_t* from = base + src * at.bytes + off;
  uint8_t* to = base + dst * at.bytes + off;
  const int n = (int)min((int64_t)kPiece, at.bytes - off);
  constexpr int kEach = kPiece / (16 * kMoveThreads);
  mx_u4 w[kEach];
  if (n == kPiece) {
#pragma unroll
    for (int e = 0; e < kEach; e++) w[e] = *(const mx_u4*)(from + (e * kMoveThreads + threadIdx.x) * 16);
#pragma unroll
    for (int e = 0; e < kEach; e++) *(mx_u4*)(to + (e * kMoveThreads + threadIdx.x) * 16) = w[e];
  } else {
    for (int o = threadIdx.x * 16; o < n; o += kMoveThreads * 16) *(mx_u4*)(to + o) = *(const mx_u4*)(from + o);
  }
  if (off == 0) {
    uint8_t* sc = keys ? at.ks : at.vs;
    for (int h = threadIdx.x; h < at.heads; h += kMoveThreads) sc[dst * at.heads + h] = sc[src * at.heads + h];
  }
}

// Table rows of the children, then the copies.
__global__ __launch_bounds__(kMoveThreads) void fork_apply(ForkArgs a, int64_t row_blocks) {
  if ((int64_t)blockIdx.x < row_blocks) {
    const int64_t per = (a.new_width + kRows - 1) / kRows, i = blockIdx.x / per, j0 = (blockIdx.x - i * per) * kRows;
    const Child c = child_of(a, i);
    const int64_t start = a.start[i] >> 1, copy = a.start[i] & 1, found = *a.found;
    const int32_t* from = a.table + (c.parent < 0 ? 0 : c.parent) * a.width;
    int32_t* to = a.new_table + i * a.new_width;
    for (int64_t j = j0 + threadIdx.x; j < min(a.new_width, j0 + kRows); j += kMoveThreads) {
      int64_t e = -1, k = -1;
      if (j < c.had - copy) {
        e = from[j];
        e = e >= 0 && e < a.n_pages ? e : -1;
      } else if (j < c.need) {
        k = start + j - (c.had - copy);
      }
      if (k >= 0 && k < found) e = a.fresh[k];
      to[j] = (int32_t)e;
    }
    return;
  }
  const int64_t all = (int64_t)a.n_layers * a.pieces, items = *a.n_copies * all;
  for (int64_t x = blockIdx.x - row_blocks; x < items; x += gridDim.x - row_blocks) {
    const int64_t i = x / all;
    move_piece(a.layers, a.pieces, (int)(x - i * all), a.src[i], a.fresh[a.dst[i]]);
  }
}

// ---------------------------------------------------------------- compact
constexpr int kChunk = 4096;  // pages of a workgroup
constexpr int kEach = kChunk / 256;

// pages in use in each chunk
__global__ __launch_bounds__(256) void compact_count(CompactArgs a, Layers l) {
  __shared__ int lds[4];
  const int64_t p0 = blockIdx.x * (int64_t)kChunk;
  int live = 0;
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    const int64_t p = p0 + e * 256 + threadIdx.x;
    live += p < a.n_pages && a.refs[p] > 0;
  }
  int all;
  (void)scan_before<256>(live, lds, &all);
  if (threadIdx.x == 0) a.count[blockIdx.x] = all;
  if (blockIdx.x == 0 && threadIdx.x == 64) put_layers(a.layers, l);
}

// Where each page goes: with L pages in use, the k-th of those at or behind L
// goes to the k-th free one before L.
__global__ __launch_bounds__(256) void compact_plan(CompactArgs a) {
  __shared__ int lds[4];
  const int tid = threadIdx.x;
  const int64_t chunks = (a.n_pages + kChunk - 1) / kChunk, me = blockIdx.x;
  int mine = 0, rest = 0;
  for (int64_t c = tid; c < chunks; c += 256) {
    const int n = a.count[c];
    (c < me ? mine : rest) += n;
  }
  int before, L;
  (void)scan_before<256>(mine, lds, &before);
  (void)scan_before<256>(rest, lds, &L);
  L += before;
  // pages in use before L: whole chunks, and the part of the chunk that holds L
  const int64_t edge = L / kChunk;
  int low = 0;
  for (int64_t c = tid; c < edge; c += 256) low += a.count[c];
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    const int64_t p = edge * kChunk + e * 256 + tid;
    low += p < L && a.refs[p] > 0;
  }
  int below;
  (void)scan_before<256>(low, lds, &below);
  // sixteen pages in a row to a thread
  const int64_t p0 = me * kChunk + tid * kEach;
  int r[kEach];
  int live = 0;
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    r[e] = p0 + e < a.n_pages ? a.refs[p0 + e] : 0;
    live += r[e] > 0;
  }
  int all;
  int64_t rank = before + scan_before<256>(live, lds, &all);  // of the thread's first page among those in use
#pragma unroll
  for (int e = 0; e < kEach; e++) {
    const int64_t p = p0 + e;
    if (p >= a.n_pages) break;
    const bool used = r[e] > 0;
    if (p < L) {
      a.place[p] = used ? (int)p : -1;
      if (!used) a.hole[p - rank] = (int)p;
    } else {
      a.place[p] = used ? -2 - (int)(rank - below) : -1;
      if (used) a.mover[rank - below] = (int)p;
    }
    rank += used;
  }
  if (me == 0 && tid == 0) {
    *a.live = L;
    *a.n_moves = L - below;
  }
}
// Both in one workgroup, the counts in LDS, where they fit: 700 pages 2.7 + 6.5 us
// for the two launches above, 6000 pages 7.6 + 9.2.
__global__ __launch_bounds__(kPlan) void compact_near(CompactArgs a, Layers l) {
  __shared__ int lds[kPlan / 64];
  __shared__ int at[kNearPages];
  const int tid = threadIdx.x, n = (int)a.n_pages;
  constexpr int kRun = 8;
  for (int p0 = 0; p0 < n; p0 += kPlan * kRun) {
    int r[kRun];
#pragma unroll
    for (int e = 0; e < kRun; e++) {
      const int p = p0 + e * kPlan + tid;
      r[e] = p < n ? a.refs[p] : 0;
    }
#pragma unroll
    for (int e = 0; e < kRun; e++) {
      const int p = p0 + e * kPlan + tid;
      if (p < n) at[p] = r[e];
    }
  }
  if (tid == 0) put_layers(a.layers, l);
  __syncthreads();
  // a run of pages to a thread, of odd length: threads' runs start in different banks
  const int run = ((n + kPlan - 1) / kPlan) | 1, p0 = min(tid * run, n), p1 = min(p0 + run, n);
  int live = 0;
  for (int p = p0; p < p1; p++) live += at[p] > 0;
  int L, below;
  int rank = scan_before<kPlan>(live, lds, &L);  // of the run's first page among those in use
  int low = 0;
  for (int p = p0; p < min(p1, L); p++) low += at[p] > 0;
  (void)scan_before<kPlan>(low, lds, &below);
  for (int p = p0; p < p1; p++) {
    const bool used = at[p] > 0;
    if (p < L) {
      at[p] = used ? p : -1;
      if (!used) a.hole[p - rank] = p;
    } else {
      at[p] = used ? -2 - (rank - below) : -1;
      if (used) a.mover[rank - below] = p;
    }
    rank += used;
  }
  if (tid == 0) {
    *a.live = L;
    *a.n_moves = L - below;
  }
  __syncthreads();
  for (int p = tid; p < n; p += kPlan) a.place[p] = at[p];
}
__device__ __forceinline__ int place_of(const CompactArgs& a, int64_t p) {
  const int at = a.place[p];
  return at < -1 ? a.hole[-2 - at] : at;
}

__global__ __launch_bounds__(kMoveThreads) void compact_apply(CompactArgs a, int64_t page_blocks, int64_t row_blocks) {
  const int64_t block = blockIdx.x;
  const int moves = *a.n_moves;
  if (block < page_blocks) {
    const int64_t L = *a.live;
    for (int64_t p = block * kRows + threadIdx.x; p < min(a.n_pages, (block + 1) * kRows); p += kMoveThreads) {
      const int to = place_of(a, p), r = a.refs[p];
      a.remap[p] = to;
      // a page in use writes its count where it goes; free ones behind the pages in
      // use, and those that leave, have 0
      if (to >= 0) a.new_refs[to] = r;
      if (p >= L) a.new_refs[p] = 0;
    }
    return;
  }
  if (block < page_blocks + row_blocks) {
    const int64_t per = (a.width + kRows - 1) / kRows, b = (block - page_blocks) / per;
    const int64_t j0 = (block - page_blocks - b * per) * kRows;
    int64_t n = a.lens[b];
    n = n < 0 ? 0 : min(n, most_tokens(a.width, a.lp));
    const int64_t held = pages_of(n, a.lp);
    for (int64_t j = j0 + threadIdx.x; j < min(a.width, j0 + kRows); j += kMoveThreads) {
      const int64_t p = j < held ? (int64_t)a.table[b * a.width + j] : -1;
      a.new_table[b * a.width + j] = p >= 0 && p < a.n_pages ? place_of(a, p) : -1;
    }
    return;
  }
  const int64_t all = (int64_t)a.n_layers * a.pieces, items = moves * all, first = page_blocks + row_blocks;
  for (int64_t x = block - first; x < items; x += gridDim.x - first) {
    const int64_t i = x / all;
    move_piece(a.layers, a.pieces, (int)(x - i * all), a.mover[i], a.hole[i]);
  }
}

Layers layers_of(const KvLayer* caches, int64_t n, int page_tokens) {
  Layers l;
  l.n = (int)std::min<int64_t>(kLayers, n);
  for (int i = 0; i < kLayers; i++) l.at[i] = PageLayer{};
  for (int i = 0; i < l.n; i++) {
    const KvLayer& c = caches[i];
    l.at[i] = PageLayer{c.kc, c.vc, c.ks, c.vs, (int64_t)c.H * page_tokens * c.D, c.H};
  }
  return l;
}
// the layers behind those that the first launch has
void put_more(PageLayer* to, const KvLayer* caches, int64_t n, int page_tokens, hipStream_t s) {
  for (int64_t c = kLayers; c < n; c += kLayers)
    hipLaunchKernelGGL(more_layers, dim3(1), dim3(1), 0, s, to + c, layers_of(caches + c, n - c, page_tokens));
}
// pieces of a page of the largest layer
int pieces_of(const KvLayer* caches, int64_t n, int page_tokens) {
  int64_t most = 0;
  for (int64_t i = 0; i < n; i++) most = std::max(most, (int64_t)caches[i].H * page_tokens * caches[i].D);
  return (int)(2 * cdiv(most, kPiece));
}
// workgroups that move pages: at most so many pieces, eight workgroups of them a compute unit
int64_t move_blocks(int64_t pages, int64_t pieces) { return std::min<int64_t>(pages * pieces, 2048); }

template <class T>
T* take(uint8_t** at, int64_t n) {
  T* p = (T*)*at;
  *at += (n * sizeof(T) + 255) / 256 * 256;
  return p;
}
int64_t most_fresh(const ForkArgs& a) {
  return std::min(a.n_pages, a.n_new * (pages_of(a.max_grow, a.lp) + 1));
}
size_t fork_layout(ForkArgs* a, uint8_t* at) {
  uint8_t* const from = at;
  a->found = take<int64_t>(&at, 1);
  a->n_copies = take<int>(&at, 1);
  a->layers = take<PageLayer>(&at, a->n_layers);
  a->children = take<int>(&at, a->n_seqs);
  a->start = take<int64_t>(&at, a->n_new);
  a->src = take<int>(&at, a->n_new);
  a->dst = take<int>(&at, a->n_new);
  a->fresh = take<int>(&at, most_fresh(*a));
  return (size_t)(at - from);
}
size_t compact_layout(CompactArgs* a, uint8_t* at) {
  uint8_t* const from = at;
  a->n_moves = take<int>(&at, 1);
  a->layers = take<PageLayer>(&at, a->n_layers);
  a->count = take<int>(&at, cdiv(a->n_pages, kChunk));
  a->place = take<int>(&at, a->n_pages);
  a->hole = take<int>(&at, a->n_pages);
  a->mover = take<int>(&at, a->n_pages);
  return (size_t)(at - from);
}

}  // namespace

// rows, pages and 2048 workgroups of moves, of 256 threads each
constexpr int64_t kMostBlocks = kMaxThreads / kMoveThreads - 2048;
bool fork_fits(const ForkArgs& a) { return a.n_new * cdiv(a.new_width, kRows) <= kMostBlocks; }
bool compact_fits(const CompactArgs& a) {
  return cdiv(a.n_pages, kRows) + a.n_seqs * cdiv(a.width, kRows) <= kMostBlocks;
}
size_t fork_workspace_bytes(ForkArgs a) { return (size_t)kCounterBytes + fork_layout(&a, nullptr); }
size_t compact_workspace_bytes(CompactArgs a) { return (size_t)kCounterBytes + compact_layout(&a, nullptr); }

hipError_t launch_fork(ForkArgs a, const KvLayer* caches, void* ws, hipStream_t s) {
  fork_layout(&a, (uint8_t*)ws + kCounterBytes);
  const int P = 1 << a.lp;
  a.pieces = pieces_of(caches, a.n_layers, P);
  const Layers first = layers_of(caches, a.n_layers, P);
  if (a.n_pages <= kNearPages) {
    hipLaunchKernelGGL(fork_plan<true>, dim3(1), dim3(kPlan), 0, s, a, first);
  } else {
    hipLaunchKernelGGL(copy_refs, dim3((unsigned)cdiv(a.n_pages, 256)), dim3(256), 0, s, a.refs, a.new_refs, a.n_pages);
    hipLaunchKernelGGL(fork_plan<false>, dim3(1), dim3(kPlan), 0, s, a, first);
  }
  if (a.n_new > 0) {
    put_more(a.layers, caches, a.n_layers, P, s);
    const int64_t rows = a.n_new * cdiv(a.new_width, kRows);
    const dim3 grid((unsigned)(rows + move_blocks(a.n_new, (int64_t)a.pieces * a.n_layers)));
    hipLaunchKernelGGL(fork_apply, grid, dim3(kMoveThreads), 0, s, a, rows);
  }
  return hipGetLastError();
}

hipError_t launch_compact(CompactArgs a, const KvLayer* caches, void* ws, hipStream_t s) {
  compact_layout(&a, (uint8_t*)ws + kCounterBytes);
  const int P = 1 << a.lp;
  a.pieces = pieces_of(caches, a.n_layers, P);
  const Layers first = layers_of(caches, a.n_layers, P);
  if (a.n_pages <= kNearPages) {
    hipLaunchKernelGGL(compact_near, dim3(1), dim3(kPlan), 0, s, a, first);
  } else {
    const unsigned chunks = (unsigned)cdiv(a.n_pages, kChunk);
    hipLaunchKernelGGL(compact_count, dim3(chunks), dim3(256), 0, s, a, first);
    hipLaunchKernelGGL(compact_plan, dim3(chunks), dim3(256), 0, s, a);
  }
  put_more(a.layers, caches, a.n_layers, P, s);
  const int64_t pages = cdiv(a.n_pages, kRows), rows = a.n_seqs * cdiv(a.width, kRows);
  const dim3 grid((unsigned)(pages + rows + move_blocks(a.n_pages / 2 + 1, (int64_t)a.pieces * a.n_layers)));
  hipLaunchKernelGGL(compact_apply, grid, dim3(kMoveThreads), 0, s, a, pages, rows);
  return hipGetLastError();
}

}  // namespace lowbit
