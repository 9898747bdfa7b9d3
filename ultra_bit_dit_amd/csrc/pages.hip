// Pages of the 8-bit cache: the next batch's tables, lengths and reference
// counts from this one's (kv8_fork), and pages in use moved together
// (kv8_compact).
//
// Everything that decides is whole numbers, and every choice goes by the order
// of children and pages, so results do not depend on the order of atomics.
// Pages are chosen by one small kernel (fork) or by chunks of 4096 pages
// (compact); their bytes are moved by a launch that fills the chip, a page's keys
// or values being one run of heads * tokens * dims bytes.
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
  const int64_t n = c.parent < 0 ? 0 : min(length_of(a, c.parent), most);
  int64_t grow = a.grow ? (int64_t)a.grow[i] : a.max_grow;
  grow = grow < 0 ? 0 : grow < a.max_grow ? grow : a.max_grow;
  c.len = min(n + grow, most);
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

// One workgroup: children of each parent, counts of holders, which tail pages
// are copied, free pages.
__global__ __launch_bounds__(kPlan) void fork_plan(ForkArgs a) {
  __shared__ int lds[kPlan / 64];
  const int tid = threadIdx.x;
  for (int64_t b = tid; b < a.n_seqs; b += kPlan) store_dev(a.children + b, 0);
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const Child c = child_of(a, i);
    if (c.tail >= 0) {
      store_dev(a.first + c.tail, INT32_MAX);
      store_dev(a.writers + c.tail, 0);
    }
  }
  meet();
  for (int64_t i = tid; i < a.n_new; i += kPlan) {
    const Child c = child_of(a, i);
    if (c.parent >= 0) add_dev(a.children + c.parent, 1);
    if (c.tail >= 0) {
      __hip_atomic_fetch_min(a.first + c.tail, (int)i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      add_dev(a.writers + c.tail, 1);
    }
  }
  meet();
  // A page loses its old holders and gains their children: nothing changes for a
  // sequence that goes on as one.  Teams of threads have a sequence each.
  int team = 64;
  while (team < kPlan && team < a.width) team *= 2;
  for (int64_t b = tid / team; b < a.n_seqs; b += kPlan / team) {
    const int64_t held = pages_of(length_of(a, b), a.lp);
    const int children = load_dev(a.children + b);
    if (children == 1 && held <= a.new_width) continue;
    for (int64_t j = tid & (team - 1); j < held; j += team) {
      const int64_t p = a.table[b * a.width + j];
      const int d = (j < a.new_width ? children : 0) - 1;
      if (d != 0 && p >= 0 && p < a.n_pages) add_dev(a.new_refs + p, d);
    }
  }
  meet();
  // pages that the children need, in their order
  int64_t total = 0;
  int copies = 0;
  for (int64_t i0 = 0; i0 < a.n_new; i0 += kPlan) {
    const int64_t i = i0 + tid;
    int need = 0, copy = 0;
    Child c;
    if (i < a.n_new) {
      c = child_of(a, i);
      // kept by the first of its writers where nobody else holds it
      copy = c.tail >= 0 && !(load_dev(a.first + c.tail) == (int)i &&
                              load_dev(a.new_refs + c.tail) == load_dev(a.writers + c.tail));
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
    }
    total += all;
    copies += all_copies;
  }
  // the first `total` free pages; the counts by wide loads, past what L1 may hold of them
  int64_t found = 0;
  constexpr int kRun = 16;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  for (int64_t p0 = 0; p0 < a.n_pages && found < total; p0 += kPlan * kRun) {
    const int64_t p = p0 + tid * kRun;
    uint32_t free = 0;
    if (p + kRun <= a.n_pages) {
      mx_u4 r[kRun / 4];
#pragma unroll
      for (int e = 0; e < kRun / 4; e++) r[e] = *(const mx_u4*)(a.new_refs + p + 4 * e);
#pragma unroll
      for (int e = 0; e < kRun; e++) free |= r[e / 4][e % 4] == 0 ? 1u << e : 0u;
    } else {
      for (int e = 0; p + e < a.n_pages; e++) free |= a.new_refs[p + e] == 0 ? 1u << e : 0u;
    }
    int all;
    int64_t at = found + scan_before<kPlan>(__builtin_popcount(free), lds, &all);
    for (; free && at < total; free &= free - 1, at++) {
      const int64_t page = p + __builtin_ctz(free);
      a.fresh[at] = (int)page;
      a.new_refs[page] = 1;
    }
    found += all;
  }
  meet();
  const bool ok = found >= total;
  for (int64_t i = tid; ok && i < copies; i += kPlan) add_dev(a.new_refs + a.src[i], -1);
  if (tid == 0) {
    *a.n_copies = ok ? copies : 0;
    *a.found = min(found, total);
    *a.failed = (int32_t)min(total - min(found, total), (int64_t)INT32_MAX);
  }
}

struct Layer {
  uint8_t *k, *v, *ks, *vs;
  int64_t bytes;  // of a page's keys
  int heads, pieces;
};
constexpr int kLayers = 32;  // of a launch
struct Layers {
  Layer at[kLayers];
  int n, pieces;  // pieces: of a page, all layers
};

// piece `piece` of page src to page dst
__device__ __forceinline__ void move_piece(const Layers& l, int piece, int64_t src, int64_t dst) {
  int i = 0;
  while (piece >= l.at[i].pieces) piece -= l.at[i++].pieces;
  const Layer& at = l.at[i];
  const int half = at.pieces / 2;
  const bool keys = piece < half;
  const int64_t off = (int64_t)(keys ? piece : piece - half) * kPiece;
  uint8_t* base = keys ? at.k : at.v;
  const uint8_t* from = base + src * at.bytes + off;
  uint8_t* to = base + dst * at.bytes + off;
  const int n = (int)min((int64_t)kPiece, at.bytes - off);
  mx_u4 w[kPiece / (16 * kMoveThreads)];
#pragma unroll
  for (int e = 0; e < kPiece / (16 * kMoveThreads); e++) {
    const int o = (e * kMoveThreads + threadIdx.x) * 16;
    if (o < n) w[e] = *(const mx_u4*)(from + o);
  }
#pragma unroll
  for (int e = 0; e < kPiece / (16 * kMoveThreads); e++) {
    const int o = (e * kMoveThreads + threadIdx.x) * 16;
    if (o < n) *(mx_u4*)(to + o) = w[e];
  }
  if (off == 0) {
    uint8_t* sc = keys ? at.ks : at.vs;
    for (int h = threadIdx.x; h < at.heads; h += kMoveThreads) sc[dst * at.heads + h] = sc[src * at.heads + h];
  }
}

// Table rows of the children, then the copies.
__global__ __launch_bounds__(kMoveThreads) void fork_apply(ForkArgs a, Layers l, int64_t row_blocks) {
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
  const int64_t items = (int64_t)*a.n_copies * l.pieces;
  for (int64_t x = blockIdx.x - row_blocks; x < items; x += gridDim.x - row_blocks) {
    const int64_t i = x / l.pieces;
    move_piece(l, (int)(x - i * l.pieces), a.src[i], a.fresh[a.dst[i]]);
  }
}

// ---------------------------------------------------------------- compact
constexpr int kChunk = 4096;  // pages of a workgroup
constexpr int kEach = kChunk / 256;

// pages in use in each chunk
__global__ __launch_bounds__(256) void compact_count(CompactArgs a) {
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
__device__ __forceinline__ int place_of(const CompactArgs& a, int64_t p) {
  const int at = a.place[p];
  return at < -1 ? a.hole[-2 - at] : at;
}

__global__ __launch_bounds__(kMoveThreads) void compact_apply(CompactArgs a, Layers l, int64_t page_blocks, int64_t row_blocks) {
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
  const int64_t items = (int64_t)moves * l.pieces, first = page_blocks + row_blocks;
  for (int64_t x = block - first; x < items; x += gridDim.x - first) {
    const int64_t i = x / l.pieces;
    move_piece(l, (int)(x - i * l.pieces), a.mover[i], a.hole[i]);
  }
}

Layers layers_of(const KvLayer* caches, int64_t n, int page_tokens) {
  Layers l;
  l.n = (int)n;
  l.pieces = 0;
  for (int i = 0; i < l.n; i++) {
    const int64_t bytes = (int64_t)caches[i].H * page_tokens * caches[i].D;
    l.at[i] = Layer{caches[i].kc, caches[i].vc, caches[i].ks, caches[i].vs, bytes, caches[i].H, (int)(2 * cdiv(bytes, kPiece))};
    l.pieces += l.at[i].pieces;
  }
  return l;
}
// workgroups that move pages: at most so many pieces, eight workgroups of them a compute unit
int64_t move_blocks(int64_t pages, const Layers& l) { return std::min<int64_t>(pages * l.pieces, 2048); }

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
  a->children = take<int>(&at, a->n_seqs);
  a->start = take<int64_t>(&at, a->n_new);
  a->src = take<int>(&at, a->n_new);
  a->dst = take<int>(&at, a->n_new);
  a->fresh = take<int>(&at, most_fresh(*a));
  a->first = take<int>(&at, a->n_pages);
  a->writers = take<int>(&at, a->n_pages);
  return (size_t)(at - from);
}
size_t compact_layout(CompactArgs* a, uint8_t* at) {
  uint8_t* const from = at;
  a->n_moves = take<int>(&at, 1);
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

hipError_t launch_fork(ForkArgs a, const KvLayer* caches, int64_t n_caches, void* ws, hipStream_t s) {
  fork_layout(&a, (uint8_t*)ws + kCounterBytes);
  hipLaunchKernelGGL(copy_refs, dim3((unsigned)cdiv(a.n_pages, 256)), dim3(256), 0, s, a.refs, a.new_refs, a.n_pages);
  hipLaunchKernelGGL(fork_plan, dim3(1), dim3(kPlan), 0, s, a);
  for (int64_t c = 0; c < n_caches && a.n_new > 0; c += kLayers) {
    const Layers l = layers_of(caches + c, std::min<int64_t>(kLayers, n_caches - c), 1 << a.lp);
    const int64_t rows = c ? 0 : a.n_new * cdiv(a.new_width, kRows);
    hipLaunchKernelGGL(fork_apply, dim3((unsigned)(rows + move_blocks(a.n_new, l))), dim3(kMoveThreads), 0, s, a, l, rows);
  }
  return hipGetLastError();
}

hipError_t launch_compact(CompactArgs a, const KvLayer* caches, int64_t n_caches, void* ws, hipStream_t s) {
  compact_layout(&a, (uint8_t*)ws + kCounterBytes);
  const unsigned chunks = (unsigned)cdiv(a.n_pages, kChunk);
  hipLaunchKernelGGL(compact_count, dim3(chunks), dim3(256), 0, s, a);
  hipLaunchKernelGGL(compact_plan, dim3(chunks), dim3(256), 0, s, a);
  for (int64_t c = 0; c < n_caches; c += kLayers) {
    const Layers l = layers_of(caches + c, std::min<int64_t>(kLayers, n_caches - c), 1 << a.lp);
    const int64_t pages = c ? 0 : cdiv(a.n_pages, kRows), rows = c ? 0 : a.n_seqs * cdiv(a.width, kRows);
    hipLaunchKernelGGL(compact_apply, dim3((unsigned)(pages + rows + move_blocks(a.n_pages / 2 + 1, l))), dim3(kMoveThreads), 0,
                       s, a, l, pages, rows);
  }
  return hipGetLastError();
}

}  // namespace lowbit
