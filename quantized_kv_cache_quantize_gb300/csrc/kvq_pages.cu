// Kernels of the paged 8-bit cache that move tokens and pages: append, copy,
// compaction (sm_103a).
#include <cuda_runtime.h>

#include "kvq_append.cuh"
#include "kvq_checks.cuh"
#include "kvq_pages.cuh"

namespace kvq {
namespace {

// ---- append ---------------------------------------------------------------
// Many new tokens.  One block per page, head and K or V, 32 values a thread in
// flight: 3 bytes of traffic per value, each value read once, its codes written
// once; the page's maximum has to be known before the first code, so the
// values wait in registers for it.  HBM bounds it, the ALU pipe is close
// behind (the maximum on pairs of values, not single ones, took 14400 tokens of
// 40 heads from 74.1 to 70.3 us, 6.3 TB/s; 4680 of 24 take 15.7 us, 5.5 TB/s).
template <int D>
__global__ void __launch_bounds__(512) append_kernel(const __grid_constant__ AppendArgs a) {
  ptx::grid_dependency_wait();
  const int kv = blockIdx.x & 1, hi_ = blockIdx.x >> 1;
  append_page<D>(a, kv, hi_ % a.p.heads, hi_ / a.p.heads);
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
  static std::atomic<int> known[64];   // by device; it does not change
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

cudaError_t launch_pages_append(const AppendArgs& a, cudaStream_t stream) {
  const bool one = a.s.offsets == nullptr;
  const long long items = one ? a.s.batch : append_items(a.s.rows, a.s.batch, a.p.shift);
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
