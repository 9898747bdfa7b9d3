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
};

// Length and new tokens of sequence b, clamped to what the table and the
// rows hold: nothing read from the device can lead outside the buffers.
struct SeqSpan {
  int64_t row0;  // first row of its new tokens
  int n, len;    // new tokens, length with them
};
__device__ __forceinline__ SeqSpan seq_span(const KvArgs& a, int64_t b) {
  SeqSpan s;
  int64_t len = a.lens[b];
  len = len < 0 ? 0 : len;
  len = len < a.max_kv ? len : a.max_kv;  // max_kv <= width * page tokens
  int64_t r0 = a.starts ? (int64_t)a.starts[b] : b * a.max_q;
  int64_t r1 = a.starts ? (int64_t)a.starts[b + 1] : r0 + a.max_q;
  r0 = r0 < 0 ? 0 : r0;
  r1 = r1 < a.total_q ? r1 : a.total_q;
  int64_t n = r1 > r0 ? r1 - r0 : 0;
  s.row0 = r0;
  s.n = (int)(n < a.max_q ? n : a.max_q);
  s.len = (int)len;
  return s;
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
  uint32_t* cnt;             // arrivals: of a group (by the place of its first share), then of a tile
};

}  // namespace lowbit
