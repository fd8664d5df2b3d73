// Host-side checks that the C ABI's entry points share.
#pragma once
#include <cstdint>
#include <cstring>
#include <utility>

#include "rn_kernels.h"

namespace rn {
namespace {

bool dtype_ok(rn_dtype d) { return d == RN_F32 || d == RN_BF16; }
int64_t size_of(rn_dtype d) { return d == RN_F32 ? 4 : d == RN_BF16 ? 2 : 1; }
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
constexpr int64_t kMaxStride = int64_t(1) << 40;

rn_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return RN_OK;
  if (!ws || have < need)
    return fail(RN_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", ws ? have : size_t(0), need);
  if (!aligned(ws, 256)) return fail(RN_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return RN_OK;
}

rn_status check_elements(const void* p, rn_dtype dt, const char* what) {
  if (!aligned(p, size_of(dt)))
    return fail(RN_ERR_INVALID_ARG, "%s must be %d-byte aligned", what, int(size_of(dt)));
  return RN_OK;
}

rn_status check_strides(const int64_t* s, const char* what) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > kMaxStride)
      return fail(RN_ERR_INVALID_ARG, "%s stride %lld outside [0, 2^40]", what, (long long)s[i]);
  return RN_OK;
}

// An output's elements must be distinct: ordered by stride, each axis has to step over all
// that the axes inside it cover.
rn_status check_distinct(const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t d, const char* what) {
  int64_t st[3] = {s[0], s[1], s[2]}, n[3] = {n0, n1, n2};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (st[j] < st[i]) { std::swap(st[i], st[j]); std::swap(n[i], n[j]); }
  __int128 span = d;   // stride * size may pass 64 bits
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) continue;
    if (st[i] < span)
      return fail(RN_ERR_INVALID_ARG, "%s: strides %lld, %lld, %lld make it overlap itself", what,
                  (long long)s[0], (long long)s[1], (long long)s[2]);
    span += static_cast<__int128>(st[i]) * (n[i] - 1);
  }
  return RN_OK;
}

// A tensor: three strided axes of elements of `es` bytes, and d contiguous ones.
struct Box {
  const void* p;
  int64_t es, s[3], n[3], d;
};

// Whether elements at i . s + [0, a.d) and diff + j . s + [0, b.d) meet, i and j inside the boxes: the
// steps k = i - j along the axes from `axis` on, ordered by falling stride, that bring diff near 0.
bool meets(int64_t diff, const Box& a, const Box& b, const int64_t* s, const int* order, int axis) {
  if (axis == 3) return diff < a.d * a.es && -diff < b.d * b.es;
  const int x = order[axis];
  const int64_t st = s[x] * a.es, up = a.n[x] - 1, down = b.n[x] - 1;
  if (st == 0) return meets(diff, a, b, s, order, axis + 1);
  const int64_t k0 = diff / st;           // (k st is at most st from diff, an address, away)
  for (int64_t k = k0 - 1; k <= k0 + 1; ++k)
    if (k <= up && -k <= down && meets(diff - k * st, a, b, s, order, axis + 1)) return true;
  return false;
}

// Whether an output overlaps another operand, as far as two tensors of one type and the same strides
// show it (of others nothing is said). The same tensor in both places is no overlap here.
bool overlaps(const Box& out, const Box& in) {
  if (!in.p || in.p == out.p || out.es != in.es) return false;
  int64_t s[3];
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    if (out.n[i] > 1 && in.n[i] > 1 && out.s[i] != in.s[i]) return false;
    s[i] = out.n[i] > 1 ? out.s[i] : in.n[i] > 1 ? in.s[i] : 0;
  }
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[order[j]] > s[order[i]]) std::swap(order[i], order[j]);
  const int64_t diff = static_cast<int64_t>(reinterpret_cast<uintptr_t>(in.p) - reinterpret_cast<uintptr_t>(out.p));
  return meets(diff, out, in, s, order, 0);
}

rn_status check_no_overlap(const Box& out, const Box& in, const char* what, const char* other) {
  if (overlaps(out, in)) return fail(RN_ERR_INVALID_ARG, "%s overlaps %s", what, other);
  return RN_OK;
}
Box box(const void* p, rn_dtype dt, const int64_t* s, int64_t n0, int64_t n1, int64_t n2, int64_t d) {
  return Box{p, size_of(dt), {s[0], s[1], s[2]}, {n0, n1, n2}, d};
}

}  // namespace
}  // namespace rn
