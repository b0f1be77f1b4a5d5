// Device helpers of the appends to the paged cache: which page a block writes,
// the scale rule over a page's new values, codes under a scale that grew.
#pragma once

#include "kvq_checks.cuh"
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

// One page of work item `item`, of one head, K or V, by a block of page * D / 32
// threads, 32 values each: they wait in registers for the page's maximum.
template <int D>
__device__ __forceinline__ void append_page(const AppendArgs& a, int kv, int head, int item) {
  constexpr int C = D / 8;             // 16-byte chunks of a row
  __shared__ uint32_t part[16];
  const int tid = threadIdx.x, lane = tid & 31;
  int b, p, r0, first, end;
  if (!append_item(a, item, b, p, r0, first, end)) return;
  const int id = seq_page(a.s, b, p, a.p.n_pages, a.status);
  if (id < 0) return;
  const int t0 = p << a.p.shift;
  const int lo = max(first - t0, 0), hi = min(end - t0, a.p.page);
  const long long blk = (long long)id * a.p.heads + head;
  if (!KVQ_IN_BOUNDS(blk, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D;
  const int c = tid % C, step = blockDim.x / C;      // page / 4 rows at a time
  const uint16_t* x = a.x[kv] + (long long)(r0 + (t0 - first)) * a.row_stride[kv] + head * a.head_stride[kv] + 8 * c;
  uint4 v[4];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = tid / C + k * step;
    v[k] = t >= lo && t < hi ? __ldg(reinterpret_cast<const uint4*>(x + t * a.row_stride[kv])) : make_uint4(0u, 0u, 0u, 0u);
  }
  const int old = lo > 0 ? scale_exp(a.p.scale[kv][blk]) : kPageExpMin;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = __vmaxu2(m, max_pair(v[k]));
  m = __reduce_max_sync(0xffffffffu, max_bits(m));
  if (blockDim.x > 32) {
    if (lane == 0) part[tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? part[lane] : 0u);
  }
  const int e = max(scale_of(m, a.status), old);
  if (lo > 0 && e > old) rescale_codes<D>(codes, lo, old - e, tid, blockDim.x);
  if (tid == 0) a.p.scale[kv][blk] = scale_bits(e);
  const float f = pow2f(-e);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = tid / C + k * step;
    if (t >= lo && t < hi) *reinterpret_cast<uint2*>(codes + t * D + 8 * c) = codes_of(v[k], f);
  }
}

}  // namespace
}  // namespace kvq
