// Device helpers of attention with shaped scores: what a row attends to.
#pragma once

#include "kvq_pages.cuh"

namespace kvq {
namespace {

// The keys [lo, hi) that a row attends to (lo >= hi: none), and the place that
// its distances are counted from: t itself, or where t lies outside its keys
// the nearest of them.  |t - j| = |ref - j| + |t - ref| for every such key, and
// the second part, the same for all, leaves the weights alone and joins lse.
struct RowView {
  int lo, hi, t, ref;
};
// row `r` of the packed tensor, at position t of sequence b
__device__ __forceinline__ RowView row_view(const PagedAttnArgs& a, int b, int r, int t, int len) {
  RowView v;
  v.t = t;
  v.hi = a.causal ? t + 1 : len;
  if (a.causal && a.shape.prefix != nullptr) v.hi = max(v.hi, __ldg(a.shape.prefix + b));
  v.lo = a.window > 0 ? t - a.window + 1 : 0;
  if (a.shape.ranges != nullptr) {
    const int2 g = __ldg(reinterpret_cast<const int2*>(a.shape.ranges) + r);
    v.lo = max(v.lo, g.x);
    v.hi = min(v.hi, g.y);
  }
  v.lo = min(max(v.lo, 0), len);
  v.hi = min(max(v.hi, 0), len);
  v.ref = v.lo < v.hi ? min(max(t, v.lo), v.hi - 1) : t;
  return v;
}
// what the distance |t - ref| takes from lse
__device__ __forceinline__ float ref_bias(const PagedAttnArgs& a, const RowView& v, int hq) {
  return a.shape.slopes == nullptr || v.t == v.ref ? 0.f : -__ldg(a.shape.slopes + hq) * (float)abs(v.t - v.ref);
}

}  // namespace
}  // namespace kvq
