// The paged 8-bit cache of keys and values (internal, not part of the public
// ABI).  Codes are e4m3; each page and head has one power of two for its keys
// and one for its values, as a byte e + 127.
//   keys   [page][head][token][dim]
//   values [page][head][dim][token]
// Values lie transposed so that the 16 tokens one lane of P V multiplies by
// are 16 contiguous bytes; keys lie as written, 16 contiguous dims per lane
// of Q K^T.
#pragma once

#include "mx.hpp"

namespace lowbit {

struct KvArgs {
  int64_t n_pages;
  int H, D, lp;              // heads, head size, log2 of the page's tokens
  uint8_t* kc;
  uint8_t* vc;
  uint8_t* ks;
  uint8_t* vs;
  int64_t n_seqs;
  const int32_t* table;      // [n_seqs][width]
  int64_t width;
  const int32_t* lens;       // tokens of each sequence, new ones included
  const int32_t* starts;     // [n_seqs + 1] rows of the new tokens, or NULL: max_q each
  int64_t total_q, max_q, max_kv;
  int32_t* bad;              // counts unreadable pages, or NULL
  // Groups in the place of sequences: a group's rows are those of its sequences.
  const int32_t* members;    // [n_seqs + 1] first sequence of each group, or NULL: member_count each
  int64_t member_count;
  int64_t n_members, member_q;  // sequences in all (0: no groups), and rows of each where `starts` (theirs) is NULL
};

// Length and new tokens of sequence b, clamped to what the table and the
// rows hold: nothing read from the device can lead outside the buffers.
struct SeqSpan {
  int64_t row0;  // first row of its new tokens
  int n, len;    // new tokens, length with them
};
// GROUPS: `a` may be of groups.
template <bool GROUPS = false>
__device__ __forceinline__ SeqSpan seq_span(const KvArgs& a, int64_t b) {
  SeqSpan s;
  int64_t len = a.lens[b];
  len = len < 0 ? 0 : len;
  len = len < a.max_kv ? len : a.max_kv;  // max_kv <= width * page tokens
  int64_t r0, r1;
  if (GROUPS && a.n_members) {
    int64_t m0 = a.members ? (int64_t)a.members[b] : b * a.member_count;
    int64_t m1 = a.members ? (int64_t)a.members[b + 1] : m0 + a.member_count;
    m0 = m0 < 0 ? 0 : m0 < a.n_members ? m0 : a.n_members;
    m1 = m1 < m0 ? m0 : m1 < a.n_members ? m1 : a.n_members;
    r0 = a.starts ? (int64_t)a.starts[m0] : m0 * a.member_q;
    r1 = a.starts ? (int64_t)a.starts[m1] : m1 * a.member_q;
  } else {
    r0 = a.starts ? (int64_t)a.starts[b] : b * a.max_q;
    r1 = a.starts ? (int64_t)a.starts[b + 1] : r0 + a.max_q;
  }
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 < a.total_q ? r1 : a.total_q;
  int64_t n = r1 > r0 ? r1 - r0 : 0;
  s.row0 = r0;
  s.n = (int)(n < a.max_q ? n : a.max_q);
  s.len = (int)len;
  return s;
}

// One layer's cache, as page moves see it.
struct KvLayer {
  int H, D;
  uint8_t *kc, *vc, *ks, *vs;
};
struct PageLayer {
  uint8_t *k, *v, *ks, *vs;
  int64_t bytes;             // of a page's keys
  int heads;
};
struct ForkArgs {
  int64_t n_pages, n_layers;
  int lp;                    // log2 of a page's tokens
  int64_t n_seqs, width;
  const int32_t* table;      // [n_seqs][width]
  const int32_t* lens;       // [n_seqs]
  const int32_t* refs;       // [n_pages] holders of each page
  int64_t n_new, new_width, max_grow;
  const int32_t* parents;    // [n_new]
  const int32_t* grow;       // [n_new] tokens to come, or NULL: max_grow each
  int32_t* new_table;        // [n_new][new_width]
  int32_t* new_lens;         // [n_new]
  int32_t* new_refs;         // [n_pages]
  int32_t* failed;           // pages that were not found
  int32_t* cut;              // children with less room than they asked for, or NULL
  int pieces;                // a page of the largest layer is moved in
  // workspace
  PageLayer* layers;
  int* children;             // [n_seqs]
  int* fresh;                // free pages, for the children in turn
  int64_t* start;            // [n_new] twice the place of a child's first one there, and 1 if that is a copy
  int *src, *dst;            // copies: a page, and the place of the one it is copied to
  int* n_copies;
  int64_t* found;            // pages in `fresh`
};
struct CompactArgs {
  int64_t n_pages, n_layers;
  int lp;
  int64_t n_seqs, width;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  int32_t* new_table;
  int32_t* new_refs;
  int32_t* remap;            // [n_pages]
  int32_t* live;             // pages in use
  int pieces;
  // workspace
  PageLayer* layers;
  int* count;                // pages in use in each chunk
  int* place;                // [n_pages] where a page goes; -2 - k: to hole[k]; -1: free
  int *hole, *mover;         // the k-th move goes from mover[k] to hole[k]
  int* n_moves;
};

// The group that sequence b belongs to, -1: none.
__device__ __forceinline__ int64_t group_of(const KvArgs& groups, int64_t b) {
  if (!groups.members) return b / groups.member_count;
  int64_t lo = 0, hi = groups.n_seqs;  // members[lo] <= b < members[hi] where b has a group
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    (groups.members[mid] <= b ? lo : hi) = mid;
  }
  return groups.members[lo] <= b && b < groups.members[lo + 1] ? lo : -1;
}

struct AttnArgs {
  KvArgs kv;
  int64_t Hq, G;
  const uint16_t* q;         // [total_q][Hq][D] bf16, q_stride elements between tokens
  int64_t q_stride;
  float scale2;              // softmax scale times log2(e)
  int causal, window;
  uint16_t* o;               // bf16, o_stride elements between tokens
  int64_t o_stride;
  float* lse;                // [total_q][Hq] or NULL
  float* part;               // results of shares: two places each, then of their groups; or of a tile's parts
  int parts;                 // of a prompt tile
  // behind shared prefixes
  KvArgs prefix;             // their groups
  int64_t group_q;           // rows of each of them to be expected; at most prefix.max_q
  float* sums;               // [parts][total_q][Hq] sums of the rows over their prefixes, before the division
  int sums_parts;            // as how many parts at most
  int whole;                 // tiles of a head whose steps are not cut into parts
  int pieces;                // of a sequence's tile, a workgroup each; kBehind: 0 for equal shares
  uint32_t* cnt;             // arrivals: of a group (by the place of its first share), then of a tile
};

// Of a call behind shared prefixes: one launch, or the groups' and the sequences'.
struct PrefixPlan {
  bool behind;               // one launch
  bool fine;                 // prompt tiles take weights in two terms
  // of that, else of the groups'.  nc 0: prompt tiles of `rows` rows in `parts` parts, the
  // first `whole` of a head uncut; else attn_decode with nc column tiles.
  int nc, rows, parts, whole;
  int64_t blocks;
  int64_t cut;               // tiles of all heads that are in parts
  int tail_nc;               // of the sequences' launch
  int64_t tail_blocks;
  int pieces;                // that a tile of attn_decode over the sequences is cut into, 0: equal shares
  size_t sums, part;         // bytes
};

}  // namespace lowbit
