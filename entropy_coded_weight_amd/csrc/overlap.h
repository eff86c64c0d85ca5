// Whether two strided tensors have a byte in common, exactly: views of one buffer may lie
// between each other (heads of a projection's rows, columns of a wider matrix) or across.
#pragma once
#include <algorithm>
#include <cstdint>
#include <utility>

namespace ecw {

// What a tensor occupies: `run` bytes, repeated along n axes, the widest stride first.
struct Box {
  static constexpr int kMost = 8;
  intptr_t at = 0;
  int n = 0;
  int64_t size[kMost], stride[kMost];  // in bytes
  int64_t run = 0;                     // 0: nothing
  bool folded = false;                 // its own elements overlap, or their order is too involved to tell

  // from there to behind the last byte, along the axes from `axis` on
  int64_t extent(int axis) const {
    int64_t e = run;
    for (int i = axis; i < n; ++i) e += (size[i] - 1) * stride[i];
    return e;
  }
};

// Of a tensor's sizes and strides in elements; strides are not negative.
inline Box box_of(const void* at, int64_t element, const int64_t* sizes, const int64_t* strides, int64_t dims) {
  Box b;
  b.at = (intptr_t)at;
  std::pair<int64_t, int64_t> axes[Box::kMost];  // stride, size
  int n = 0;
  for (int64_t i = 0; i < dims; ++i) {
    if (sizes[i] == 0) return b;
    if (sizes[i] == 1) continue;
    if (strides[i] == 0 || n == Box::kMost)
      b.folded = true;
    else
      axes[n++] = {strides[i] * element, sizes[i]};
  }
  std::sort(axes, axes + n);
  b.run = element;
  int first = 0;  // axes that follow without a gap are part of the run
  while (first < n && axes[first].first == b.run) b.run *= axes[first++].second;
  int64_t inner = b.run;
  for (int i = first; i < n; ++i) {
    b.folded |= axes[i].first < inner;
    inner += (axes[i].second - 1) * axes[i].first;
  }
  while (n > first) {
    --n;
    b.stride[b.n] = axes[n].first, b.size[b.n++] = axes[n].second;
  }
  return b;
}

// a's axes from ia on, `ahead` bytes behind b's from ib on.  The wider stride S is taken first: a
// step along it moves a by S against b, and only few such distances bring the rest of both together.
inline bool boxes_meet(const Box& a, int ia, const Box& b, int ib, int64_t ahead, int* budget) {
  if (ahead >= b.extent(ib) || -ahead >= a.extent(ia)) return false;
  if (ia == a.n && ib == b.n) return true;
  if (--*budget < 0) return true;
  const int64_t sa = ia < a.n ? a.stride[ia] : 0, sb = ib < b.n ? b.stride[ib] : 0, s = std::max(sa, sb);
  int64_t lo = 0, hi = 0;  // steps of a less steps of b
  if (sa == s) hi = a.size[ia++] - 1;
  if (sb == s) lo = 1 - b.size[ib++];
  // -extent of a < ahead + k s < extent of b
  auto below = [](int64_t p, int64_t q) { return p >= 0 ? p / q : -((-p + q - 1) / q); };  // floor
  lo = std::max(lo, below(-a.extent(ia) - ahead, s) + 1);
  hi = std::min(hi, below(b.extent(ib) - ahead - 1, s));
  for (int64_t k = lo; k <= hi; ++k)
    if (boxes_meet(a, ia, b, ib, ahead + k * s, budget)) return true;
  return false;
}
// Layouts that would take more than a few hundred steps to tell apart count as overlapping.
inline bool boxes_meet(const Box& a, const Box& b) {
  int budget = 256;
  return a.run && b.run && boxes_meet(a, 0, b, 0, a.at - b.at, &budget);
}

}  // namespace ecw
