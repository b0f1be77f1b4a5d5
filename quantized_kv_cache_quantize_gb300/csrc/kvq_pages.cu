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
  if (s.offsets == nullptr) {
    b = item;
    r0 = b;
    n = 1;
    p = 0;
  } else {
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
  return (p << a.p.shift) < end;
}

// one warp per page, head and K or V
template <int D>
__global__ void __launch_bounds__(64) append_kernel(const AppendArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31, kv = threadIdx.x >> 5;
  const int head = blockIdx.x % a.p.heads;
  int b, p, r0, first, end;
  if (!append_item(a, blockIdx.x / a.p.heads, b, p, r0, first, end)) return;
  const int id = seq_page(a.s, b, p, a.p.n_pages, a.status);
  if (id < 0) return;
  const int t0 = p << a.p.shift;
  const int lo = max(first - t0, 0), hi = min(end - t0, a.p.page);
  const long long blk = (long long)id * a.p.heads + head;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D + C * lane;
  const uint16_t* x = a.x[kv] + (r0 + (t0 - first)) * a.row_stride[kv] + head * a.head_stride[kv] + C * lane;
  float m = 0.f;
  bool fine = true;
  for (int t = lo; t < hi; ++t)
    for (int c = 0; c < C; ++c) {
      const float v = fabsf(__uint_as_float((uint32_t)__ldg(x + t * a.row_stride[kv] + c) << 16));
      m = fmaxf(m, v);
      fine &= in_code_range(v);
    }
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!fine) atomicCAS(a.status, 0, (int)KVQ_ERR_RANGE);
  int e = exp_for_max(m);
  if (lo > 0) {
    const int old = scale_exp(a.p.scale[kv][blk]);
    if (e > old) {
      const float f = pow2f(old - e);
      for (int t = 0; t < lo; ++t)
        for (int c = 0; c < C; c += 2) {
          const uint32_t h = f16x2_of_e4m3x2(*reinterpret_cast<uint16_t*>(codes + t * D + c));
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
          *reinterpret_cast<uint16_t*>(codes + t * D + c) = (uint16_t)e4m3x4(v.x * f, v.y * f, 0.f, 0.f);
        }
    }
    e = max(e, old);
  }
  __syncwarp();
  if (lane == 0) a.p.scale[kv][blk] = scale_bits(e);
  const float f = pow2f(-e);
  for (int t = lo; t < hi; ++t)
    for (int c = 0; c < C; c += 2) {
      const float v0 = __uint_as_float((uint32_t)__ldg(x + t * a.row_stride[kv] + c) << 16);
      const float v1 = __uint_as_float((uint32_t)__ldg(x + t * a.row_stride[kv] + c + 1) << 16);
      *reinterpret_cast<uint16_t*>(codes + t * D + c) = (uint16_t)e4m3x4(v0 * f, v1 * f, 0.f, 0.f);
    }
}

// ---- copies ---------------------------------------------------------------

// one page of one layer, by all threads of the block
__device__ __forceinline__ void copy_page(const PagePool& p, int layer, int src, int dst) {
  const long long from = (long long)layer * p.n_pages + src, to = (long long)layer * p.n_pages + dst;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint4* s = reinterpret_cast<const uint4*>(p.codes[kv] + from * p.page_bytes);
    uint4* d = reinterpret_cast<uint4*>(p.codes[kv] + to * p.page_bytes);
    for (long long i = threadIdx.x; i < p.page_bytes / 16; i += blockDim.x) d[i] = s[i];
    for (int h = threadIdx.x; h < p.heads; h += blockDim.x)
      p.scale[kv][to * p.heads + h] = p.scale[kv][from * p.heads + h];
  }
}

// (src, dst) pairs as kernel parameters: no upload, and nothing that must
// outlive the call
constexpr int kCopyPairs = 448;
struct CopyArgs {
  PagePool pool;
  int n;
  int32_t src[kCopyPairs], dst[kCopyPairs];
};

__global__ void __launch_bounds__(256) copy_kernel(const __grid_constant__ CopyArgs a) {
  for (long long i = blockIdx.x; i < (long long)a.n * a.pool.layers; i += gridDim.x) {
    const int pair = (int)(i % a.n);
    copy_page(a.pool, (int)(i / a.n), a.src[pair], a.dst[pair]);
  }
}

// ---- compaction -------------------------------------------------------------
// The plan, one block: a bitmap of the live pages in shared memory, the number
// of live pages below each of its words, then holes and movers paired by rank.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int warp_sum[kPlanThreads / 32];
  const int n_pages = a.pool.n_pages, words = (n_pages + 31) / 32;
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < words; i += kPlanThreads) bits[i] = 0u;
  __syncthreads();
  const long long total = (long long)a.batch * a.width;
  for (long long i = tid; i < total; i += kPlanThreads) {
    const int id = __ldg(a.table + (i / a.width) * a.stride + i % a.width);
    if (id >= n_pages) page_error(a.status);
    if (id >= 0 && id < n_pages) atomicOr(bits + (id >> 5), 1u << (id & 31));
  }
  __syncthreads();
  // each thread's run of words, and the live pages before it
  const int per = (words + kPlanThreads - 1) / kPlanThreads;
  const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int mine = 0;
  for (int w = w0; w < w1; ++w) mine += __popc(bits[w]);
  int incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[tid >> 5] = incl;
  __syncthreads();
  int before = incl - mine, n_live = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < (tid >> 5)) before += warp_sum[w];
    n_live += warp_sum[w];
  }
  int32_t* src = a.ws + 4;
  int32_t* dst = src + n_pages;
  int32_t* to = dst + n_pages;
  // holes below n_live, by rank (ids before it that are not live)
  int live = before;
  for (int w = w0; w < w1; ++w) {
    const uint32_t v = bits[w];
    for (uint32_t h = ~v; h != 0u; h &= h - 1u) {
      const int bit = __ffs((int)h) - 1, id = 32 * w + bit;
      if (id < n_live) dst[id - (live + __popc(v & ((1u << bit) - 1u)))] = id;
    }
    live += __popc(v);
  }
  // live pages below n_live, and so the rank of the first mover
  __shared__ int kept;
  if (tid == 0) kept = 0;
  __syncthreads();
  int below = 0;
  for (int w = w0; w < w1; ++w) {
    const int id = 32 * w;
    const uint32_t m = id + 32 <= n_live ? ~0u : id >= n_live ? 0u : (1u << (n_live - id)) - 1u;
    below += __popc(bits[w] & m);
  }
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0 && below != 0) atomicAdd(&kept, below);
  __syncthreads();
  live = before;
  for (int w = w0; w < w1; ++w) {
    const uint32_t v = bits[w];
    for (uint32_t h = v; h != 0u; h &= h - 1u) {
      const int bit = __ffs((int)h) - 1, id = 32 * w + bit;
      if (id >= n_live) {
        const int rank = live + __popc(v & ((1u << bit) - 1u)) - kept;
        src[rank] = id;
        to[id] = dst[rank];
      }
    }
    live += __popc(v);
  }
  if (tid == 0) {
    a.ws[0] = n_live - kept;
    *a.n_live = n_live;
  }
}

__global__ void __launch_bounds__(256) compact_apply_kernel(const CompactArgs a) {
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
  for (long long i = blockIdx.x; i < (long long)moves * a.pool.layers; i += gridDim.x) {
    const int k = (int)(i % moves);
    copy_page(a.pool, (int)(i / moves), src[k], dst[k]);
  }
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
  const long long items = a.s.offsets == nullptr ? a.s.batch : (a.s.rows >> a.p.shift) + 2LL * a.s.batch;
  const long long grid = items * a.p.heads;
  if (grid == 0) return cudaSuccess;
  if (a.p.d == 64) append_kernel<64><<<(unsigned)grid, 64, 0, stream>>>(a);
  else append_kernel<128><<<(unsigned)grid, 64, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
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
    long long grid = (long long)a.n * p.layers;
    if (grid > 8LL * sms) grid = 8LL * sms;
    copy_kernel<<<(unsigned)grid, 256, 0, stream>>>(a);
    note_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int smem = (a.pool.n_pages + 31) / 32 * 4;
  cudaError_t e = ensure_smem_limit(compact_plan_kernel, kCompactMaxPages / 8, g_plan_smem);
  if (e != cudaSuccess) return e;
  compact_plan_kernel<<<1, kPlanThreads, smem, stream>>>(a);
  note_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  compact_apply_kernel<<<(unsigned)(8 * sms), 256, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace kvq
