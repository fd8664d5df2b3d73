// Batches of sequences as the calls over prompts get them: padded (a row of the tensors each, of which
// a length is used) or packed end to end. Blocks take `len` token rows of one sequence.
#pragma once
#include <algorithm>

#include "rn_device.h"

namespace rn {

struct Seqs {
  int32_t S, N;               // sequences; most tokens of one
  int64_t T;                  // packed rows, 0 for a padded batch
  int32_t len, n_seg;         // rows a block takes; such pieces of a padded row
  const int32_t* cu;
  const int32_t* lens;
};

// Pieces of all sequences. Packed, sequence s starting at row r has the pieces from r / len + s on up to
// the next one's first: at least as many as its rows need, and one if it has none. Sequence S stands
// for the rows behind the last one.
__host__ __device__ inline int64_t seq_pieces(const Seqs& q) {
  return q.T > 0 ? q.T / q.len + q.S + 1 : static_cast<int64_t>(q.S) * q.n_seg;
}
inline void seq_cut(Seqs* q, int len) {
  q->len = len;
  q->n_seg = (q->N + len - 1) / len;
}
// The pieces along the grid's y and z axes, with x blocks each.
inline dim3 seq_grid(const Seqs& q, int64_t x) {
  const int64_t all = seq_pieces(q), y = std::min<int64_t>(all, 65535);
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y), static_cast<unsigned>((all + y - 1) / y));
}

// One sequence, whatever the device arrays hold: never outside the tensors.
struct Span {
  int s;                      // sequence (S: none)
  int piece;                  // piece of it
  int len;                    // its tokens
  int64_t row0;               // packed: its first token row; padded: 0
  int64_t own;                // its rows
};
__device__ __forceinline__ int64_t seq_first(const Seqs& q, int s) {
  return min(max(static_cast<int64_t>(q.cu[s]), int64_t(0)), q.T);
}
__device__ __forceinline__ void seq_span(const Seqs& q, int s, Span* p) {
  p->s = s;
  if (q.T > 0) {
    const int64_t b = seq_first(q, s);
    const int64_t e = s >= q.S ? q.T : max(seq_first(q, s + 1), b);
    p->row0 = b;
    p->own = e - b;
    p->len = s >= q.S ? 0 : static_cast<int>(min(e - b, static_cast<int64_t>(q.N)));
  } else {
    p->row0 = 0;
    p->own = q.N;
    p->len = q.lens ? min(max(q.lens[s], 0), q.N) : q.N;
  }
}
// The sequence and piece number w stands for; false if there is none. All lanes of a wave call it.
__device__ __forceinline__ bool seq_place(const Seqs& q, int64_t w, Span* p) {
  if (q.T == 0) {
    const int64_t s = w / q.n_seg;
    if (s >= q.S) return false;
    seq_span(q, static_cast<int>(s), p);
    p->piece = static_cast<int>(w - s * q.n_seg);
    return true;
  }
  // the last sequence whose first piece is at most w, a lane a candidate
  auto first = [&](int s) { return seq_first(q, s) / q.len + s; };
  int lo = 0;
  for (int n = q.S + 1; n > 1;) {
    const int each = (n + 63) / 64, at = static_cast<int>(threadIdx.x & 63) * each;
    const int k = 63 - __clzll(__ballot(at < n && first(lo + at) <= w) | 1);
    lo += k * each;
    n = min(each, n - k * each);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int64_t piece = w - first(lo);
  seq_span(q, lo, p);
  p->piece = static_cast<int>(piece);
  return piece >= 0 && piece * q.len < max(p->own, int64_t(1));
}
// Offset of token 0 of the sequence in a tensor with strides (sequence, ..., token).
__device__ __forceinline__ int64_t seq_base(const Seqs& q, const Span& p, int64_t seq_stride, int64_t tok_stride) {
  return q.T > 0 ? p.row0 * tok_stride : p.s * seq_stride;
}
// Index of the state of sequence s in the caller's buffers, or -1.
__device__ __forceinline__ int seq_slot(const int32_t* slots, int n_slots, int s) {
  if (!slots) return s;
  const int x = slots[s];
  return x >= 0 && x < n_slots ? x : -1;
}

}  // namespace rn
