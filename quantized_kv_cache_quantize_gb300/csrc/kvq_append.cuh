// Device helpers of the appends to the paged cache: which page a block writes,
// the scale rule over a page's new values, codes under a scale that grew.
#pragma once

#include "kvq_pages.cuh"

namespace kvq {
namespace {

// Work item: one page that some sequence writes.  Sequence b's items start at
// offsets[b] / page + 2 b: its n rows touch at most n / page + 2 pages, and
// floors of the cumulative count leave at least n / page.  The items of all
// sequences are then below rows / page + 2 batch, known on the host.
__device__ __forceinline__ bool append_item(const AppendArgs& a, int item, int& b, int& p, int& r0,
                                            int& first, int& end) {
  const PageSeqs& s = a.s;
  int n;
  {
    int lo = 0, hi = s.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((max(__ldg(s.offsets + mid), 0) >> a.p.shift) + 2 * mid <= item) lo = mid; else hi = mid - 1;
    }
    b = lo;
    seq_rows(s, b, r0, n, a.status);
    p = item - ((max(__ldg(s.offsets + b), 0) >> a.p.shift) + 2 * b);
    if (n == 0 || p < 0) return false;
  }
  const int len = seq_len(s, b, a.p.shift, a.status);
  const int start = len - n;
  if (start < 0) page_error(a.status);      // more new tokens than the length holds
  first = max(start, 0);
  end = len;
  r0 += first - start;                      // row of token `first`
  p += first >> a.p.shift;
  return p <= (end - 1) >> a.p.shift;       // (end may be 0)
}

// Earlier codes [row][D] of rows [0, lo) under a scale grown by 2^-shift
// (shift < 0), by the threads of the block.
template <int D>
__device__ __forceinline__ void rescale_codes(uint8_t* codes, int lo, int shift, int tid, int threads) {
  const float f = pow2f(shift);
  uint2* c = reinterpret_cast<uint2*>(codes);
  for (int i = tid; i < lo * (D / 8); i += threads) {
    uint2 w = c[i];
    uint32_t* v = &w.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t a = f16x2_of_e4m3x2((uint16_t)v[k]), b = f16x2_of_e4m3x2((uint16_t)(v[k] >> 16));
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
      v[k] = e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
    }
    c[i] = w;
  }
}

// largest magnitudes of 8 BF16 values, those of even and odd ones, as their
// bits (they order like the values; an infinity or a NaN comes out above every
// finite number)
__device__ __forceinline__ uint32_t max_pair(const uint4& v) {
  constexpr uint32_t k = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
}
__device__ __forceinline__ uint32_t max_bits(uint32_t pair) { return max(pair & 0xffffu, pair >> 16); }
__device__ __forceinline__ uint2 codes_of(const uint4& v, float f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t o[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    o[k] = e4m3x4(__uint_as_float(w[2 * k] << 16) * f, __uint_as_float(w[2 * k] & 0xffff0000u) * f,
                  __uint_as_float(w[2 * k + 1] << 16) * f, __uint_as_float(w[2 * k + 1] & 0xffff0000u) * f);
  return make_uint2(o[0], o[1]);
}
// the largest value of the block that the scale rule sees: beyond the code
// range (or not finite) it is recorded and the codes saturate
__device__ __forceinline__ int scale_of(float m, int* status) {
  if (!in_code_range(m)) {
    atomicCAS(status, 0, (int)KVQ_ERR_RANGE);
    return kPageExpMax;
  }
  return exp_for_max(m);
}
__device__ __forceinline__ int scale_of(uint32_t bits, int* status) { return scale_of(__uint_as_float(bits << 16), status); }

}  // namespace
}  // namespace kvq
