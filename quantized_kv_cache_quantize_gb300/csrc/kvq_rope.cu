// Rotary positions: the table, the rotation of queries and keys, and the append
// to the paged cache that rotates its keys on the way (sm_103a).
#include <cuda_runtime.h>

#include "kvq_append.cuh"
#include "kvq_checks.cuh"
#include "kvq_pages.cuh"
#include "kvq_rope.cuh"

namespace kvq {
namespace {

// ---- the table --------------------------------------------------------------
struct FillArgs {
  float2* cs;
  int n, pairs;
  double factor;
  double f[kRopeMaxPairs];
};
// Angles, cosines and sines in 64 bits, once for the life of a table.
__global__ void __launch_bounds__(256) rope_fill_kernel(const __grid_constant__ FillArgs a) {
  ptx::grid_dependency_wait();
  const long long total = (long long)a.n * a.pairs;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const int p = (int)(i % a.pairs);
    double s, c;
    sincos((double)(i / a.pairs) * a.f[p], &s, &c);
    a.cs[i] = make_float2((float)(a.factor * c), (float)(a.factor * s));
  }
}

// ---- rotation ---------------------------------------------------------------
// A thread rotates 16 channels of one row and head.
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const unsigned units = (unsigned)a.d / 16u;
  const int heads = a.x[0].heads + a.x[1].heads;
  unsigned long long i = (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int u = (int)(i % units);
  i /= units;
  const int row = (int)(i % (unsigned)a.rows);
  i /= (unsigned)a.rows;
  int h = (int)(i % (unsigned)heads);
  const unsigned long long b = i / (unsigned)heads;
  if (b >= (unsigned long long)a.batch) return;
  const bool second = h >= a.x[0].heads;
  if (second) h -= a.x[0].heads;
  const RopeTensor& x = a.x[second ? 1 : 0];
  int c0, c1;
  rope_chunks(a.t, u, c0, c1);
  const uint16_t* from = x.x + (long long)b * x.xb + (long long)row * x.xr + (long long)h * x.xh;
  uint16_t* to = x.y + (long long)b * x.yb + (long long)row * x.yr + (long long)h * x.yh;
  uint4 v = *reinterpret_cast<const uint4*>(from + c0), w = *reinterpret_cast<const uint4*>(from + c1);
  if (u < (a.t.pairs >> 3)) {
    const RopeAt at = rope_at(a.t, a.pos + (long long)b * a.pb + (long long)row * a.pr, a.pa, a.status);
    float2 cs[8];
    rope_turn<8>(a.t, at, 8 * u, a.inverse != 0, cs);
    rope_apply(a.t, cs, v, w);
  }
  *reinterpret_cast<uint4*>(to + c0) = v;
  *reinterpret_cast<uint4*>(to + c1) = w;
}

// ---- append -----------------------------------------------------------------
// the sequence of packed row r, by its offsets
__device__ __forceinline__ int seq_of_row(const PageSeqs& s, int r) {
  int lo = 0, hi = s.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(s.offsets + mid) <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Queries beside the append: 16 channels of one row and head a thread.
template <int D>
__device__ __forceinline__ void append_query(const AppendRopeArgs& p, unsigned long long i) {
  const PageSeqs& s = p.a.s;
  constexpr unsigned kUnits = D / 16;
  const int u = (int)(i % kUnits);
  i /= kUnits;
  const int h = (int)(i % (unsigned)p.q.heads);
  const unsigned long long row = i / (unsigned)p.q.heads;
  if (row >= (unsigned long long)s.rows) return;
  const int r = (int)row;
  if (s.offsets != nullptr && (r < __ldg(s.offsets) || r >= __ldg(s.offsets + s.batch))) return;
  int c0, c1;
  rope_chunks(p.t, u, c0, c1);
  const uint16_t* from = p.q.x + (long long)r * p.q.xr + (long long)h * p.q.xh;
  uint16_t* to = p.q.y + (long long)r * p.q.yr + (long long)h * p.q.yh;
  uint4 v = *reinterpret_cast<const uint4*>(from + c0), w = *reinterpret_cast<const uint4*>(from + c1);
  if (u < (p.t.pairs >> 3)) {
    RopeAt at;
    if (p.pos != nullptr) {
      at = rope_at(p.t, p.pos + (long long)r * p.pr, 1, p.a.status);
    } else {
      int b = r, end = r + 1;
      if (s.offsets != nullptr) {
        b = seq_of_row(s, r);
        end = __ldg(s.offsets + b + 1);
      }
      at = rope_at(p.t, seq_len(s, b, p.a.p.shift, p.a.status) - (end - r), p.a.status);
    }
    float2 cs[8];
    rope_turn<8>(p.t, at, 8 * u, false, cs);
    rope_apply(p.t, cs, v, w);
  }
  *reinterpret_cast<uint4*>(to + c0) = v;
  *reinterpret_cast<uint4*>(to + c1) = w;
}

// Chunk c (8 channels) of a key row, rotated, in fp32.  The lanes of a row's
// D / 8 chunks are neighbours; every lane of the warp calls.
template <int D>
__device__ __forceinline__ void rotate_chunk(const RopeTab& t, const RopeAt& at, int c, bool live, const uint4& v,
                                             float (&f)[8]) {
  floats_of(v, f);
  const int p8 = t.pairs >> 3;
  if (t.interleaved) {
    if (c < 2 * p8 && live) {
      float2 cs[4];
      rope_turn<4>(t, at, 4 * c, false, cs);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = f[2 * k], x1 = f[2 * k + 1];
        f[2 * k] = turn_first(x0, x1, cs[k]);
        f[2 * k + 1] = turn_second(x0, x1, cs[k]);
      }
    }
    return;
  }
  const int other = c < p8 ? c + p8 : c < 2 * p8 ? c - p8 : c;
  const int lane = (int)(threadIdx.x & 31), from = lane - c % (D / 8) + other;
  uint4 o;
  o.x = __shfl_sync(0xffffffffu, v.x, from);
  o.y = __shfl_sync(0xffffffffu, v.y, from);
  o.z = __shfl_sync(0xffffffffu, v.z, from);
  o.w = __shfl_sync(0xffffffffu, v.w, from);
  if (c < 2 * p8 && live) {
    float g[8];
    floats_of(o, g);
    float2 cs[8];
    rope_turn<8>(t, at, 8 * (c < p8 ? c : c - p8), false, cs);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = c < p8 ? turn_first(f[k], g[k], cs[k]) : turn_second(g[k], f[k], cs[k]);
  }
}

__device__ __forceinline__ uint32_t max_abs_bits(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float f) {
  return make_uint2(e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f), e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
}

// Many new tokens: a block per page, head and K or V; behind them blocks of
// query rows.
template <int D>
__global__ void __launch_bounds__(512) append_rope_kernel(const __grid_constant__ AppendRopeArgs p, unsigned kv_blocks) {
  constexpr int C = D / 8;             // 16-byte chunks of a row
  __shared__ uint32_t part[16];
  const AppendArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31;
  ptx::grid_dependency_wait();
  if (blockIdx.x >= kv_blocks) {
    append_query<D>(p, (unsigned long long)(blockIdx.x - kv_blocks) * blockDim.x + tid);
    return;
  }
  const int kv = blockIdx.x & 1, hi_ = blockIdx.x >> 1;
  const int head = hi_ % a.p.heads;
  int b, pg, r0, first, end;
  if (!append_item(a, hi_ / a.p.heads, b, pg, r0, first, end)) return;
  const int id = seq_page(a.s, b, pg, a.p.n_pages, a.status);
  if (id < 0) return;
  const int t0 = pg << a.p.shift;
  const int lo = max(first - t0, 0), hi = min(end - t0, a.p.page);
  const long long blk = (long long)id * a.p.heads + head;
  if (!KVQ_IN_BOUNDS(blk, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D;
  const int c = tid % C, step = blockDim.x / C;      // page / 4 rows at a time
  const int row = r0 + (t0 - first);                 // packed row of the page's token 0
  const uint16_t* x = a.x[kv] + (long long)row * a.row_stride[kv] + head * a.head_stride[kv] + 8 * c;
  float f[4][8];
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = tid / C + k * step;
    const bool live = t >= lo && t < hi;
    const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(x + t * a.row_stride[kv])) : make_uint4(0u, 0u, 0u, 0u);
    if (kv == 0) {
      RopeAt at{};
      if (live)
        at = p.pos != nullptr ? rope_at(p.t, p.pos + (long long)(row + t) * p.pr, 1, a.status)
                              : rope_at(p.t, t0 + t, a.status);
      rotate_chunk<D>(p.t, at, c, live, v, f[k]);
    } else {
      floats_of(v, f[k]);
    }
  }
  const int old = lo > 0 ? scale_exp(a.p.scale[kv][blk]) : kPageExpMin;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = max(m, max_abs_bits(f[k]));
  m = __reduce_max_sync(0xffffffffu, m);
  if (blockDim.x > 32) {
    if (lane == 0) part[tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? part[lane] : 0u);
  }
  const int e = max(scale_of(__uint_as_float(m), a.status), old);
  if (lo > 0 && e > old) rescale_codes<D>(codes, lo, old - e, tid, blockDim.x);
  if (tid == 0) a.p.scale[kv][blk] = scale_bits(e);
  const float s = pow2f(-e);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int t = tid / C + k * step;
    if (t >= lo && t < hi) *reinterpret_cast<uint2*>(codes + t * D + 8 * c) = codes_of(f[k], s);
  }
}

// One token of every sequence: a warp per sequence, head and K or V, as in the
// plain append; behind them warps of query rows.
template <int D>
__global__ void __launch_bounds__(128) append_one_rope_kernel(const __grid_constant__ AppendRopeArgs p, unsigned kv_blocks) {
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  if (blockIdx.x >= kv_blocks) {
    append_query<D>(p, (unsigned long long)(blockIdx.x - kv_blocks) * blockDim.x + threadIdx.x);
    return;
  }
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1), head = (int)((w >> 1) % a.p.heads);
  const long long item = (w >> 1) / a.p.heads;
  if (item >= a.s.batch) return;
  const int b = (int)item;
  const bool has = lane < D / 8;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (has) v = __ldg(reinterpret_cast<const uint4*>(a.x[kv] + b * a.row_stride[kv] + head * a.head_stride[kv] + 8 * lane));
  const int len = seq_len(a.s, b, a.p.shift, a.status);
  if (len < 1) {
    page_error(a.status);     // a new token, but no place for it
    return;
  }
  const int pg = (len - 1) >> a.p.shift, t = (len - 1) & (a.p.page - 1);
  const int id = seq_page(a.s, b, pg, a.p.n_pages, a.status);
  if (id < 0) return;
  const long long blk = (long long)id * a.p.heads + head;
  if (!KVQ_IN_BOUNDS(blk, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D;
  const int old = t > 0 ? scale_exp(a.p.scale[kv][blk]) : kPageExpMin;
  float f[8];
  if (kv == 0) {
    const RopeAt at = p.pos != nullptr ? rope_at(p.t, p.pos + (long long)b * p.pr, 1, a.status)
                                       : rope_at(p.t, len - 1, a.status);
    rotate_chunk<D>(p.t, at, lane % (D / 8), has, v, f);
  } else {
    floats_of(v, f);
  }
  const uint32_t m = __reduce_max_sync(0xffffffffu, max_abs_bits(f));
  const int e = max(scale_of(__uint_as_float(m), a.status), old);
  if (t > 0 && e > old) rescale_codes<D>(codes, t, old - e, lane, 32);
  if (lane == 0 && (t == 0 || e > old)) a.p.scale[kv][blk] = scale_bits(e);
  if (has) *reinterpret_cast<uint2*>(codes + t * D + 8 * lane) = codes_of(f, pow2f(-e));
}

}  // namespace

cudaError_t launch_rope_fill(float* cos_sin, int n, int pairs, const double* frequency, double factor,
                             cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  FillArgs f{};
  f.cs = reinterpret_cast<float2*>(cos_sin);
  f.n = n;
  f.pairs = pairs;
  f.factor = factor;
  for (int p = 0; p < pairs; ++p) f.f[p] = frequency[p];
  const long long blocks = ((long long)n * pairs + 255) / 256, most = 16LL * sms;
  return launch_dependent(rope_fill_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, stream, f);
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
  const long long threads = (long long)a.batch * a.rows * (a.x[0].heads + a.x[1].heads) * (a.d / 16);
  return launch_dependent(rope_kernel, (unsigned)((threads + 255) / 256), 256, 0, stream, a);
}

cudaError_t launch_pages_append_rope(const AppendRopeArgs& p, cudaStream_t stream) {
  const AppendArgs& a = p.a;
  const bool one = a.s.offsets == nullptr;
  const long long items = one ? a.s.batch : (a.s.rows >> a.p.shift) + 2LL * a.s.batch;
  const long long units = items * a.p.heads * 2;
  const int threads = one ? 128 : a.p.page * a.p.d / 32;
  const long long kv_blocks = one ? (units + 3) / 4 : units;
  const long long q_blocks = ((long long)a.s.rows * p.q.heads * (a.p.d / 16) + threads - 1) / threads;
  if (kv_blocks + q_blocks == 0) return cudaSuccess;
  const auto kern = one ? (a.p.d == 64 ? append_one_rope_kernel<64> : append_one_rope_kernel<128>)
                        : (a.p.d == 64 ? append_rope_kernel<64> : append_rope_kernel<128>);
  return launch_dependent(kern, (unsigned)(kv_blocks + q_blocks), threads, 0, stream, p, (unsigned)kv_blocks);
}

}  // namespace kvq
