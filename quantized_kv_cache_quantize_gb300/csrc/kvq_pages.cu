// Kernels of the paged 8-bit cache that move tokens and pages: append, copy,
// compaction (sm_103a).
#include <cuda_runtime.h>

#include "kvq_checks.cuh"
#include "kvq_pages.cuh"

namespace kvq {
namespace {

// ---- append ---------------------------------------------------------------
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
__device__ __forceinline__ int scale_of(uint32_t bits, int* status) {
  const float m = __uint_as_float(bits << 16);
  if (!in_code_range(m)) {
    atomicCAS(status, 0, (int)KVQ_ERR_RANGE);
    return kPageExpMax;
  }
  return exp_for_max(m);
}

// Many new tokens.  One block per page, head and K or V, 32 values a thread in
// flight: 3 bytes of traffic per value, each value read once, its codes written
// once; the page's maximum has to be known before the first code, so the
// values wait in registers for it.  HBM bounds it, the ALU pipe is close
// behind (the maximum on pairs of values, not single ones, took 14400 tokens of
// 40 heads from 74.1 to 70.3 us, 6.3 TB/s; 4680 of 24 take 15.7 us, 5.5 TB/s).
template <int D>
__global__ void __launch_bounds__(512) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int C = D / 8;             // 16-byte chunks of a row
  __shared__ uint32_t part[16];
  const int tid = threadIdx.x, lane = tid & 31;
  ptx::grid_dependency_wait();
  const int kv = blockIdx.x & 1, hi_ = blockIdx.x >> 1;
  const int head = hi_ % a.p.heads;
  int b, p, r0, first, end;
  if (!append_item(a, hi_ / a.p.heads, b, p, r0, first, end)) return;
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

// One token of every sequence: a warp per sequence, head and K or V, D / 8
// lanes of it with values.  What counts is the chain of dependent loads:
// length, table entry, then scale and row together.
template <int D>
__global__ void __launch_bounds__(128) append_one_kernel(const __grid_constant__ AppendArgs a) {
  const int lane = threadIdx.x & 31;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
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
  const int p = (len - 1) >> a.p.shift, t = (len - 1) & (a.p.page - 1);
  const int id = seq_page(a.s, b, p, a.p.n_pages, a.status);
  if (id < 0) return;
  const long long blk = (long long)id * a.p.heads + head;
  if (!KVQ_IN_BOUNDS(blk, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D;
  const int old = t > 0 ? scale_exp(a.p.scale[kv][blk]) : kPageExpMin;
  const uint32_t m = __reduce_max_sync(0xffffffffu, max_bits(max_pair(v)));
  const int e = max(scale_of(m, a.status), old);
  if (t > 0 && e > old) rescale_codes<D>(codes, t, old - e, lane, 32);
  if (lane == 0 && (t == 0 || e > old)) a.p.scale[kv][blk] = scale_bits(e);
  if (has) *reinterpret_cast<uint2*>(codes + t * D + 8 * lane) = codes_of(v, pow2f(-e));
}

// ---- copies ---------------------------------------------------------------

// Copies, bound by HBM (each byte read and written once).  The unit of work is
// 32 KB of one page's K or V in one layer, eight 16-byte loads a thread in
// flight before the first store, so that the blocks of one resident wave
// finish together whatever the number of pages (whole pages a block left a
// fifth of the wave idle at 495 pages x 8 layers: 176 us).
constexpr int kCopyThreads = 256, kCopyVecs = 8, kCopyUnit = kCopyThreads * kCopyVecs;   // in 16-byte vectors
__host__ __device__ __forceinline__ long long copy_units(const PagePool& p, long long pages) {
  const long long segs = (p.page_bytes / 16 + kCopyUnit - 1) / kCopyUnit;
  return pages * p.layers * 2 * segs;
}
// unit u of `n` pages: pages in the order pair(k, &src, &dst)
template <typename Pair>
__device__ __forceinline__ void copy_unit(const PagePool& p, long long u, int n, Pair pair) {
  const int segs = (int)((p.page_bytes / 16 + kCopyUnit - 1) / kCopyUnit);
  const int seg = (int)(u % segs);
  u /= segs;
  const int kv = (int)(u & 1);
  u >>= 1;
  int src, dst;
  pair((int)(u % n), &src, &dst);
  const long long layer = u / n;
  const long long from = layer * p.n_pages + src, to = layer * p.n_pages + dst;
  const uint4* s = reinterpret_cast<const uint4*>(p.codes[kv] + from * p.page_bytes);
  uint4* d = reinterpret_cast<uint4*>(p.codes[kv] + to * p.page_bytes);
  const int end = (int)(p.page_bytes / 16), at = seg * kCopyUnit + threadIdx.x;
  uint4 v[kCopyVecs];
#pragma unroll
  for (int k = 0; k < kCopyVecs; ++k)
    if (at + k * kCopyThreads < end) v[k] = s[at + k * kCopyThreads];
#pragma unroll
  for (int k = 0; k < kCopyVecs; ++k)
    if (at + k * kCopyThreads < end) d[at + k * kCopyThreads] = v[k];
  if (seg == 0)
    for (int h = threadIdx.x; h < p.heads; h += kCopyThreads)
      p.scale[kv][to * p.heads + h] = p.scale[kv][from * p.heads + h];
}

// (src, dst) pairs as kernel parameters: no upload, and nothing that must
// outlive the call
constexpr int kCopyPairs = 448;
struct CopyArgs {
  PagePool pool;
  int n;
  int32_t src[kCopyPairs], dst[kCopyPairs];
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  ptx::grid_dependency_wait();
  const long long total = copy_units(a.pool, a.n);
  for (long long u = blockIdx.x; u < total; u += gridDim.x)
    copy_unit(a.pool, u, a.n, [&](int k, int* src, int* dst) {
      *src = a.src[k];
      *dst = a.dst[k];
    });
}

// ---- compaction -------------------------------------------------------------
// The plan, one block: a bitmap of the live pages in shared memory and the
// number of live pages below every eighth of its words; with those any page's
// rank is a few loads away, and holes and movers are paired by rank, a page a
// thread.  What it takes is latency (a walk over the bits of a word by one
// thread took 11.5 us for 2000 pages).
constexpr int kPlanThreads = 1024, kRankWords = 8;
__host__ __device__ __forceinline__ int plan_words(int n_pages) {
  return ((n_pages + 31) / 32 + kRankWords - 1) / kRankWords * kRankWords;
}
__host__ __device__ __forceinline__ int plan_bytes(int n_pages) {
  return plan_words(n_pages) * 4 + plan_words(n_pages) / kRankWords * 4;
}
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ CompactArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int warp_sum[kPlanThreads / 32];
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int n_pages = a.pool.n_pages, words = plan_words(n_pages), groups = words / kRankWords;
  int* below = reinterpret_cast<int*>(bits + words);   // [groups] live pages before the group
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < words; i += kPlanThreads) bits[i] = 0u;
  __syncthreads();
  const long long total = (long long)a.batch * a.width;
#pragma unroll 4
  for (long long i = tid; i < total; i += kPlanThreads) {
    const int id = __ldg(a.table + (i / a.width) * a.stride + i % a.width);
    if (id >= n_pages) page_error(a.status);
    if (id >= 0 && id < n_pages) atomicOr(bits + (id >> 5), 1u << (id & 31));
  }
  __syncthreads();
  // each thread's run of groups, and the live pages before it
  const int per = (groups + kPlanThreads - 1) / kPlanThreads;
  const int g0 = min(tid * per, groups), g1 = min(g0 + per, groups);
  int mine = 0;
  for (int w = g0 * kRankWords; w < g1 * kRankWords; ++w) mine += __popc(bits[w]);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[tid >> 5] = incl;
  __syncthreads();
  int all = warp_sum[lane];                // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += v;
  }
  const int n_live = __shfl_sync(0xffffffffu, all, 31);
  int before = __shfl_sync(0xffffffffu, all, (tid >> 5) - 1 & 31);
  before = (tid < 32 ? 0 : before) + incl - mine;
  for (int g = g0; g < g1; ++g) {
    below[g] = before;
    for (int w = g * kRankWords; w < (g + 1) * kRankWords; ++w) before += __popc(bits[w]);
  }
  __syncthreads();
  auto rank = [&](int id) {                // live pages below id (id < 32 * words)
    const int w = id >> 5;
    int r = below[w / kRankWords] + __popc(bits[w] & ((1u << (id & 31)) - 1u));
    for (int k = w & ~(kRankWords - 1); k < w; ++k) r += __popc(bits[k]);
    return r;
  };
  auto live = [&](int id) { return ((bits[id >> 5] >> (id & 31)) & 1u) != 0u; };
  int32_t* src = a.ws + 4;
  int32_t* dst = src + n_pages;
  int32_t* to = dst + n_pages;
  const int kept = n_live < n_pages ? rank(n_live) : n_live;
  for (int id = tid; id < n_live; id += kPlanThreads)
    if (!live(id)) dst[id - rank(id)] = id;
  __syncthreads();
  for (int id = n_live + tid; id < n_pages; id += kPlanThreads)
    if (live(id)) {
      const int r = rank(id) - kept, into = dst[r];
      src[r] = id;
      to[id] = into;
    }
  if (tid == 0) {
    a.ws[0] = n_live - kept;
    *a.n_live = n_live;
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(const __grid_constant__ CompactArgs a) {
  ptx::grid_dependency_wait();
  const int n_pages = a.pool.n_pages;
  const int moves = a.ws[0], n_live = *a.n_live;
  const int32_t* src = a.ws + 4;
  const int32_t* dst = src + n_pages;
  const int32_t* to = dst + n_pages;
  const long long total = (long long)a.batch * a.width;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / a.width, col = i % a.width;
    const int id = a.table[row * a.stride + col];
    a.table_out[row * a.out_stride + col] = id >= n_live && id < n_pages ? to[id] : id;
  }
  const long long units = copy_units(a.pool, moves);
  for (long long u = blockIdx.x; u < units; u += gridDim.x)
    copy_unit(a.pool, u, moves, [&](int k, int* from, int* into) {
      *from = src[k];
      *into = dst[k];
    });
}

std::atomic<uint64_t> g_plan_smem{0};

}  // namespace

int sm_count_current() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

cudaError_t launch_pages_append(const AppendArgs& a, cudaStream_t stream) {
  const bool one = a.s.offsets == nullptr;
  const long long items = one ? a.s.batch : (a.s.rows >> a.p.shift) + 2LL * a.s.batch;
  const long long units = items * a.p.heads * 2;
  if (units == 0) return cudaSuccess;
  if (one) {
    const unsigned grid = (unsigned)((units + 3) / 4);
    return a.p.d == 64 ? launch_dependent(append_one_kernel<64>, grid, 128, 0, stream, a)
                       : launch_dependent(append_one_kernel<128>, grid, 128, 0, stream, a);
  }
  const int threads = a.p.page * a.p.d / 32;
  return a.p.d == 64 ? launch_dependent(append_kernel<64>, (unsigned)units, threads, 0, stream, a)
                     : launch_dependent(append_kernel<128>, (unsigned)units, threads, 0, stream, a);
}

cudaError_t launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  CopyArgs a;
  a.pool = p;
  for (int at = 0; at < n; at += kCopyPairs) {
    a.n = n - at < kCopyPairs ? n - at : kCopyPairs;
    for (int i = 0; i < a.n; ++i) {
      a.src[i] = src[at + i];
      a.dst[i] = dst[at + i];
    }
    const long long units = copy_units(p, a.n), most = 8LL * sms;
    const cudaError_t e = launch_dependent(copy_kernel, (unsigned)(units < most ? units : most), kCopyThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int smem = plan_bytes(a.pool.n_pages);
  cudaError_t e = ensure_smem_limit(compact_plan_kernel, plan_bytes(kCompactMaxPages), g_plan_smem);
  if (e != cudaSuccess) return e;
  e = launch_dependent(compact_plan_kernel, 1u, kPlanThreads, smem, stream, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(compact_apply_kernel, (unsigned)(8 * sms), kCopyThreads, 0, stream, a);
}

}  // namespace kvq
