// Linear attention with a decay per head and token: what its kernels share.
#pragma once
#include "rn_kernels.h"

namespace rn {

// Where a kernel starts and ends: a whole sequence; the state a segment adds on its own
// (first pass over a sequence cut into segments); the outputs of a segment whose starting
// state the scan left in the workspace (third pass). Where the sequences' lengths are not known
// and most may be of one segment (`flat`), the third pass is of the first kind: it takes such
// sequences whole, and the other two leave them out.
enum LinMode : int { kLinWhole = 0, kLinState = 1, kLinOut = 2 };

struct LinArgs {
  int32_t S, N, H, Hq, Hk, Hv, dk, dv;
  int32_t n_slots;
  int32_t seg_len, n_seg;     // tokens a segment (a multiple of 64), most segments a sequence
  int64_t T;                  // packed rows, 0 for a padded batch
  float scale;
  bool zero_rest;
  bool flat;                  // blocks along a packed batch's segments, not sequences x n_seg
  int64_t qs[3], ks[3], vs[3], gs[3], os[3];
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* slots;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* state_in;
  float* state_out;
  void* out;
  float* seg_state;           // [segments][H][dk][dv]
  float* seg_decay;           // [segments][H]
};

// First token row (packed), number of tokens, and number of rows of sequence s, whatever the
// device arrays hold: never outside the tensors. Sequence S of a packed batch is the rows
// behind the last one.
__device__ __forceinline__ void lin_span(const LinArgs& a, int s, int64_t* row0, int* len, int64_t* own) {
  if (a.T > 0) {
    const int64_t b = min(max(static_cast<int64_t>(a.cu[s]), int64_t(0)), a.T);
    const int64_t e = s == a.S ? a.T : min(max(static_cast<int64_t>(a.cu[s + 1]), b), a.T);
    *row0 = b;
    *own = e - b;
    *len = s == a.S ? 0 : static_cast<int>(min(e - b, static_cast<int64_t>(a.N)));
  } else {
    *row0 = 0;
    *own = a.N;
    *len = a.lens ? min(max(a.lens[s], 0), a.N) : a.N;
  }
}
// Offset of the sequence's first token in a tensor with strides st (head and token aside).
__device__ __forceinline__ int64_t lin_base(const LinArgs& a, const int64_t* st, int s, int64_t row0) {
  return a.T > 0 ? row0 * st[2] : s * st[0];
}
// Head and column slice of a block. Blocks are dealt to the 8 XCDs, each with an L2 of its own,
// by their number modulo 8: the slices of a head, and heads that share q and k, come at
// distances of the number of such groups, so that (with 8 groups or a multiple) they meet in
// one L2 and q and k reach it once.
__device__ __forceinline__ void lin_block(const LinArgs& a, int x, int* h, int* slice) {
  const int groups = min(a.Hq, a.Hk), each = a.H / groups;
  const int g = x % groups, rest = x / groups;
  *slice = rest / each;
  *h = g * each + (rest - *slice * each);
}
// Index of the state of sequence s in the caller's buffers, or -1.
__device__ __forceinline__ int lin_slot(const LinArgs& a, int s) {
  if (!a.slots) return s;
  const int x = a.slots[s];
  return x >= 0 && x < a.n_slots ? x : -1;
}
// Row of segment g of sequence s in the workspace: distinct for all segments, and below
// total_segments() whatever the device arrays hold. In a flat grid only sequences of more than one
// segment use it, and one that starts at token row r owns 2r/L on: with n tokens, n > L, that is
// 2n/L rows (rounded down) at least, and ceil(n/L) of them are needed.
__device__ __forceinline__ int64_t lin_segment(const LinArgs& a, int s, int64_t row0, int g) {
  return a.flat ? 2 * row0 / a.seg_len + g : static_cast<int64_t>(s) * a.n_seg + g;
}
// The last of the sequences 0 .. S of a packed batch that a predicate holds for, which holds up to
// one of them (whatever it says, one of them): a lane a candidate.
template <class F>
__device__ __forceinline__ int lin_last(const LinArgs& a, F holds) {
  int lo = 0;
  for (int n = a.S + 1; n > 1;) {
    const int each = (n + 63) / 64, at = static_cast<int>(threadIdx.x & 63) * each;
    const int k = 63 - __clzll(__ballot(at < n && holds(lo + at)) | 1);
    lo += k * each;
    n = min(each, n - k * each);
  }
  return lo;
}
__device__ __forceinline__ int64_t lin_first(const LinArgs& a, int s) {
  return min(max(static_cast<int64_t>(a.cu[s]), int64_t(0)), a.T);
}
// The segment and sequence of a block. In a flat grid, sequence s, starting at row r, has the blocks
// from r/L + s on up to the next one's first. False: none.
__device__ __forceinline__ bool lin_place(const LinArgs& a, int* s, int* seg) {
  if (!a.flat) {
    *s = blockIdx.z;
    *seg = blockIdx.y;
    return true;
  }
  const int64_t w = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  auto first = [&](int i) { return lin_first(a, i) / a.seg_len + i; };
  const int lo = lin_last(a, [&](int i) { return first(i) <= w; });
  const int64_t g = w - first(lo);
  *s = lo;
  *seg = static_cast<int>(g);
  return g >= 0;                // (past the sequence's tokens: rows to be zeroed, or nothing)
}
// The grid of a pass, with x blocks along heads and columns; `rest`: for the rows behind a packed
// batch's last sequence too.
inline dim3 lin_grid(const LinArgs& a, int x, bool rest) {
  if (!a.flat) return dim3(x, a.n_seg, a.S + (rest ? 1 : 0));
  const int64_t all = a.T / a.seg_len + a.S + 1, y = all < 65535 ? all : 65535;
  return dim3(x, static_cast<unsigned>(y), static_cast<unsigned>((all + y - 1) / y));
}
// Zeros into the columns [c0, c0 + nc) of head h in the rows of sequence s behind its tokens
// (flag RN_LINEAR_ZERO_REST); the blocks of its segments share them.
template <int OUT>
__device__ __forceinline__ void lin_zero_rest(const LinArgs& a, int s, int g, int h, int c0, int nc,
                                              int64_t row0, int len, int64_t own) {
  const int64_t base = (a.T > 0 ? row0 * a.os[2] : s * a.os[0]) + h * a.os[1] + c0;
  const int64_t blocks = a.flat ? (row0 + own) / a.seg_len - row0 / a.seg_len + 1 : a.n_seg;
  const int64_t step = blocks * a.seg_len;
  for (int64_t t0 = len + static_cast<int64_t>(g) * a.seg_len; t0 < own; t0 += step) {
    const int64_t n = min(own - t0, static_cast<int64_t>(a.seg_len)) * nc;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
      Elem<OUT>::store(a.out, base + (t0 + i / nc) * a.os[2] + i % nc, 0.f);
  }
}

// Matrix-core kernel (bf16 in and out, whole 16-byte rows).
int lin_mfma_blocks(const LinArgs& a);     // blocks a sequence and segment takes
hipError_t launch_lin_mfma(const LinArgs& a, LinMode mode, hipStream_t st);

}  // namespace rn
