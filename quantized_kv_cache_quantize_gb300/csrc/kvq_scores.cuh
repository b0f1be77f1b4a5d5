// Device helpers of attention with shaped scores: what a row attends to, and the
// shaping itself.
//
// Numbers.  A capped score is cap * tanh(x), x the score over the cap.  For |x| <=
// 1, where scores that a cap is meant for lie, tanh is x times a polynomial in x^2
// (tanh_fit.py), 2^-22 of it at most with its roundings: products on pairs, none of
// them on the special-function unit, which the softmax's exponentials need.  Beyond,
// 1 - 2 / (1 + 2^(2 x log2 e)): two special functions a score, off by 2^-22; one and
// a half in far_scores, which takes one reciprocal for two.  A distance is a whole
// number, exact in fp32 up to 2^24.
#pragma once

#include <math_constants.h>

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

constexpr int kPlain = 0, kBiased = 1, kCapped = 2;   // kernels' modes; a capped one may be biased too

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// the smaller, or NaN where one is
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// tanh of a pair, |x| <= 1
__device__ __forceinline__ uint64_t tanh_small(uint64_t x) {
  auto both = [](float c) { return ptx::f2_pack(c, c); };
  const uint64_t z = ptx::f2_mul(x, x);
  uint64_t p = ptx::f2_fma(z, both(1.038025133e-03f), both(-6.194324698e-03f));
  p = ptx::f2_fma(p, z, both(2.027970739e-02f));
  p = ptx::f2_fma(p, z, both(-5.345164612e-02f));
  p = ptx::f2_fma(p, z, both(1.332507581e-01f));
  p = ptx::f2_fma(p, z, both(-3.333282769e-01f));
  p = ptx::f2_fma(p, z, both(9.999999404e-01f));
  return ptx::f2_mul(p, x);
}
// tanh of any number, given tanh_small of it
__device__ __forceinline__ float tanh_any(float x, float small) {
  const float far = fmaf(-2.f, rcp_approx(1.f + ptx::ex2_approx(2.885390082f * x)), 1.f);
  return fabsf(x) <= 1.f ? small : far;
}

// What shapes the scores of one row, in units of log 2.
struct RowShape {
  float cap2;      // cap log2 e
  float slope2;    // slope log2 e
  bool biased;     // of the call
};
template <int MODE>
__device__ __forceinline__ RowShape row_shape(const PagedAttnArgs& a, int hq) {
  RowShape r;
  r.cap2 = MODE == kCapped ? a.shape.cap * 1.4426950408889634f : 0.f;
  r.biased = a.shape.slopes != nullptr;
  r.slope2 = r.biased ? __ldg(a.shape.slopes + hq) * 1.4426950408889634f : 0.f;
  return r;
}
// the factor of a raw score: to units of log 2, or of the cap
template <int MODE>
__device__ __forceinline__ float raw_factor(const PagedAttnArgs& a) {
  return MODE == kCapped ? a.scale / a.shape.cap : a.scale * 1.4426950408889634f;
}

// Up to 0.4 of the cap four terms do, and fold with what follows: with the cap in
// the coefficients the shaped score in units of log 2 is x (c0 + c1 x^2 + c2 x^4 +
// c3 x^6), x the score over the cap, its last product the one that also adds what
// stands in the exponent beside it: five products on pairs more than a plain score
// has, where the seven terms take nine (24 heads of 4680 rows, 23400 keys: 1.33
// against 1.67 ms).  (The row's and page's factor ck must stay
// out of the coefficients: raw scores of codes reach 1.5e7, ck 3e-8 where x is still
// 0.4, and a c3 that holds ck^7 is lost to fp32's range, 2^-14 of the cap.)
constexpr float kLowX = 0.4f;
struct LowCap {
  float c0, c1, c2, c3;
};
__device__ __forceinline__ LowCap low_cap(float cap2) {
  return LowCap{9.999998808e-01f * cap2, -3.333135545e-01f * cap2, 1.327087432e-01f * cap2, -4.754934832e-02f * cap2};
}
// of raw scores s times ck
__device__ __forceinline__ uint64_t low_scores(uint64_t s, float ck, const LowCap& c, uint64_t beside) {
  auto both = [](float x) { return ptx::f2_pack(x, x); };
  const uint64_t x = ptx::f2_mul(s, both(ck)), z = ptx::f2_mul(x, x);
  uint64_t p = ptx::f2_fma(both(c.c3), z, both(c.c2));
  p = ptx::f2_fma(p, z, both(c.c1));
  p = ptx::f2_fma(p, z, both(c.c0));
  return ptx::f2_fma(p, x, beside);
}

// The same for any score, by cap2 (1 - 2 / (1 + t)), t = 2^(2 x log2 e), alone: off
// by 2^-20 of the cap at most, whatever the score (2 r, r = 1 / (1 + t) <= 1, with
// five roundings of 2^-24 or 2^-23, t off by 2^-21 where it counts).  Half the
// instructions of the choice between two ways (cap_block), and little that a weight
// in FP16 shows while the cap is below kShortCap: 2^-12 there, half its rounding.
// ct: 2 ck log2 e.
constexpr float kShortCap = 256.f;
__device__ __forceinline__ uint64_t far_scores(uint64_t s, float ct, uint64_t minus2cap, uint64_t cap_beside) {
  float x0, x1;
  ptx::f2_unpack(ptx::f2_mul(s, ptx::f2_pack(ct, ct)), x0, x1);
  // (1 / a, 1 / b) = (b, a) / (a b): one reciprocal for two.  Past 2^60 1 / a is
  // nothing beside 1, and a b stays in fp32.  (A NaN takes its neighbour with it.)
  const float e0 = ptx::ex2_approx(min_nan(x0, 60.f)), e1 = ptx::ex2_approx(min_nan(x1, 60.f));
  ptx::f2_unpack(ptx::f2_add(ptx::f2_pack(e0, e1), ptx::f2_pack(1.f, 1.f)), x0, x1);
  const float r = rcp_approx(x0 * x1);
  return ptx::f2_fma(ptx::f2_mul(ptx::f2_pack(x1, x0), ptx::f2_pack(r, r)), minus2cap, cap_beside);
}

// What is left to do to a shaped score: a factor to units of log 2.
template <int MODE>
__device__ __forceinline__ float shape_factor(const RowShape& r, float ck) {
  return r.biased ? 1.f : MODE == kCapped ? r.cap2 : ck;
}
// tanh of 16 raw scores times ck, in place
__device__ __forceinline__ void cap_block(uint32_t* s, float ck) {
  const uint64_t c2 = ptx::f2_pack(ck, ck);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint64_t x2 = ptx::f2_mul(ptx::f2_pack(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), c2);
    float x0, y0, x, y;
    ptx::f2_unpack(x2, x0, y0);
    ptx::f2_unpack(tanh_small(x2), x, y);
    s[2 * k] = __float_as_uint(tanh_any(x0, x));
    s[2 * k + 1] = __float_as_uint(tanh_any(y0, y));
  }
}
// The bias of 16 neighbouring keys, key 0 `dist` before the row's reference
// place, added to their scores times f.
__device__ __forceinline__ void bias_block(uint32_t* s, float f, const RowShape& r, int dist) {
  const float d0 = (float)dist;
#pragma unroll
  for (int k = 0; k < 16; ++k)
    s[k] = __float_as_uint(fmaf(-r.slope2, fabsf(d0 - (float)k), __uint_as_float(s[k]) * f));
}

}  // namespace
}  // namespace kvq
