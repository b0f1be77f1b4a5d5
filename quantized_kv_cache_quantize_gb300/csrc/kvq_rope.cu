// Rotary positions: the table, the rotation of queries and keys, and the append
// to the paged cache that rotates its keys on the way (sm_103a).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

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
// A block per R rows and eight heads of one tensor.  Each value is read and
// written once and HBM bounds the large sizes; the turns, 4 bytes a channel, would
// double the reads if every head fetched its own.  Queries and keys of 4680 tokens,
// 24 heads, in the window's layout: 22.4 us, 5.1 TB/s (four heads a thread in
// flight and three blocks an SM 25.2 us, five blocks 27.7).  R = 4 spreads a small
// call over the SMs: 64 rows of 40 heads take 4.1 us, all of it latency.
template <int D, int R, bool INTER>
__global__ void __launch_bounds__(256, 4) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float4 turns[R * kRopeRow];
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const unsigned tiles = ((unsigned)a.rows + R - 1) / R;
  const unsigned q_groups = ((unsigned)a.x[0].heads + kRopeHeads - 1) / kRopeHeads,
                 groups = q_groups + ((unsigned)a.x[1].heads + kRopeHeads - 1) / kRopeHeads;
  unsigned g = blockIdx.x % groups;
  const unsigned rest = blockIdx.x / groups;
  const int row0 = (int)(rest % tiles) * R;
  const long long b = rest / tiles;
  const bool second = g >= q_groups;
  if (second) g -= q_groups;
  RopeTensor x = a.x[0];
  if (second) x = a.x[1];
  const int h0 = (int)g * kRopeHeads, rows = min(R, a.rows - row0), heads = min(kRopeHeads, x.heads - h0);
  if (!KVQ_IN_BOUNDS(b * a.rows + row0 + rows - 1, (long long)a.batch * a.rows, a.status, a.bounds_site) ||
      !KVQ_IN_BOUNDS(h0 + heads - 1, x.heads, a.status, a.bounds_site))
    return;
  const int32_t* pos = a.pos + b * a.pb + row0 * a.pr;
  rope_tile<D, R, (R + 7) / 8, INTER>(a.t, a.inverse != 0, turns, rows, heads,
                  x.x + b * x.xb + row0 * x.xr + h0 * x.xh, x.xr, x.xh, x.y + b * x.yb + row0 * x.yr + h0 * x.yh, x.yr,
                  x.yh, a.status, a.bounds_site, [&](int r, int axis) { return __ldg(pos + r * a.pr + axis * a.pa); });
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

// Queries beside the append, R rows and eight heads: block `at` of theirs.
template <int D, int R, int N, bool INTER>
__device__ __forceinline__ void append_queries(const AppendRopeArgs& p, unsigned at, float4* turns) {
  const PageSeqs& s = p.a.s;
  const unsigned groups = ((unsigned)p.q.heads + kRopeHeads - 1) / kRopeHeads;
  const int h0 = (int)(at % groups) * kRopeHeads;
  int row0 = (int)(at / groups) * R, end = min(row0 + R, s.rows);
  if (s.offsets != nullptr) {   // rows that no sequence has are left alone
    row0 = max(row0, __ldg(s.offsets));
    end = min(end, __ldg(s.offsets + s.batch));
  }
  if (row0 >= end) return;
  const int heads = min(kRopeHeads, p.q.heads - h0);
  if (!KVQ_IN_BOUNDS(row0, end, p.a.status, p.a.bounds_site) || !KVQ_IN_BOUNDS(end - 1, s.rows, p.a.status, p.a.bounds_site) ||
      !KVQ_IN_BOUNDS(h0 + heads - 1, p.q.heads, p.a.status, p.a.bounds_site))
    return;
  auto place = [&](int r, int axis) {
    if (p.pos != nullptr) return __ldg(p.pos + (row0 + r) * p.pr + axis);
    int b = row0 + r, next = b + 1;
    if (s.offsets != nullptr) {
      b = seq_of_row(s, b);
      next = __ldg(s.offsets + b + 1);
    }
    const int at = seq_len(s, b, p.a.p.shift, p.a.status) - (next - (row0 + r));
    if (at < 0) page_error(p.a.status);   // a row before its sequence's first token
    return max(at, 0);
  };
  rope_tile<D, R, N, INTER>(p.t, false, turns, end - row0, heads, p.q.x + row0 * p.q.xr + h0 * p.q.xh,
                  p.q.xr, p.q.xh, p.q.y + row0 * p.q.yr + h0 * p.q.yh, p.q.yr, p.q.yh, p.a.status, p.a.bounds_site, place);
}

// largest magnitude of m and 16 values, a NaN before all
__device__ __forceinline__ float most_of(float m, const float (&f)[8], const float (&g)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f[k]), "f"(g[k]));
  return m;
}
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float f) {
  const uint64_t f2 = ptx::f2_pack(f, f);
  float x[8];
#pragma unroll
  for (int k = 0; k < 8; k += 2) ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(v[k], v[k + 1]), f2), x[k], x[k + 1]);
  return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}

// One page of keys, heads [h0, h1), by a block of page * D / 32 threads: two units
// of 16 channels a thread and head.  The page's turns go to shared memory once
// for all heads; the next head's values are on their way while this one's page
// maximum is found.
template <int D, bool INTER>
__device__ __forceinline__ void append_keys(const AppendRopeArgs& p, int item, int h0, int h1, float4* turns) {
  constexpr int U = D / 16;
  __shared__ uint32_t part[2][16];
  const AppendArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, step = blockDim.x / U;   // half a page of rows
  int b, pg, r0, first, end;
  if (!append_item(a, item, b, pg, r0, first, end)) return;
  const int id = seq_page(a.s, b, pg, a.p.n_pages, a.status);
  if (id < 0) return;
  const int t0 = pg << a.p.shift;
  const int lo = max(first - t0, 0), hi = min(end - t0, a.p.page);
  if (!KVQ_IN_BOUNDS((long long)id * a.p.heads + h1 - 1, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  const long long row = r0 + (t0 - first);           // packed row of the page's token 0
  if (lo < hi && (!KVQ_IN_BOUNDS(row + lo, a.s.rows, a.status, a.bounds_site) ||
                  !KVQ_IN_BOUNDS(row + hi - 1, a.s.rows, a.status, a.bounds_site)))
    return;
  const int u = tid % U;
  int c0, c1;
  rope_chunks(p.t, u, c0, c1);
  const uint16_t* x = a.x[0] + row * a.row_stride[0];
  uint4 v[2], w[2];
  auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = tid / U + k * step;
      const uint16_t* from = x + t * a.row_stride[0] + h * a.head_stride[0];
      const bool live = t >= lo && t < hi;
      v[k] = live ? __ldg(reinterpret_cast<const uint4*>(from + c0)) : make_uint4(0u, 0u, 0u, 0u);
      w[k] = live ? __ldg(reinterpret_cast<const uint4*>(from + c1)) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  load(h0);
  rope_stage(p.t, turns, hi - lo, false, a.status, a.bounds_site, [&](int r, int axis) {
    return p.pos != nullptr ? __ldg(p.pos + (row + lo + r) * p.pr + axis) : t0 + lo + r;
  });
  __syncthreads();
  for (int h = h0; h < h1; ++h) {
    const long long blk = (long long)id * a.p.heads + h;
    uint8_t* codes = a.p.codes[0] + blk * a.p.page * D;
    const int old = lo > 0 ? scale_exp(a.p.scale[0][blk]) : kPageExpMin;
    float f[2][8], g[2][8];
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = tid / U + k * step;
      if (u < (p.t.pairs >> 3) && t >= lo && t < hi) {
        float4 cs[4];
        rope_entries(turns + (t - lo) * kRopeRow, u, cs);
        rope_apply<INTER>(p.t, cs, v[k], w[k], f[k], g[k]);
      } else {
        floats_of(v[k], f[k]);
        floats_of(w[k], g[k]);
      }
      most = most_of(most, f[k], g[k]);
    }
    if (h + 1 < h1) load(h + 1);
    uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (blockDim.x > 32) {   // (two buffers: a head's is read while the next one's is written)
      uint32_t* mine = part[(h - h0) & 1];
      if (lane == 0) mine[tid >> 5] = m;
      __syncthreads();
      m = __reduce_max_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? mine[lane] : 0u);
    }
    const int e = max(scale_of(__uint_as_float(m), a.status), old);
    if (lo > 0 && e > old) rescale_codes<D>(codes, lo, old - e, tid, blockDim.x);
    if (tid == 0) a.p.scale[0][blk] = scale_bits(e);
    const float s = pow2f(-e);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int t = tid / U + k * step;
      if (t >= lo && t < hi) {
        *reinterpret_cast<uint2*>(codes + t * D + c0) = codes_of(f[k], s);
        *reinterpret_cast<uint2*>(codes + t * D + c1) = codes_of(g[k], s);
      }
    }
  }
}

// Many new tokens: blocks of keys (a page and `heads` heads), of query rows, of
// values (a page and head), the longest first.  Bound by HBM, 5 bytes of K and V a
// channel and 4 of the queries, with the ALU pipe behind it (every product and sum
// of the rotation by itself).  4680 tokens of 24 heads and their queries: 5.0 TB/s;
// two heads a block of keys 37.4 us, four 33.4, eight 30.5, queries behind the
// values 3 us more; without the load of the next head ahead 0.5 us more.
struct AppendGrid {
  unsigned k_blocks, q_blocks;
  int heads;    // per block of keys
  int q_rows;   // per block of query rows
};
template <int D, bool INTER>
__global__ void __launch_bounds__(512, 2) append_rope_kernel(const __grid_constant__ AppendRopeArgs p, const AppendGrid g) {
  extern __shared__ float4 turns[];
  ptx::grid_dependency_wait();
  unsigned at = blockIdx.x;
  if (at < g.k_blocks) {
    const unsigned groups = (unsigned)(p.a.p.heads + g.heads - 1) / (unsigned)g.heads;
    const int h0 = (int)(at % groups) * g.heads;
    append_keys<D, INTER>(p, (int)(at / groups), h0, min(h0 + g.heads, p.a.p.heads), turns);
    return;
  }
  at -= g.k_blocks;
  if (at < g.q_blocks) {
    if (g.q_rows == 16) append_queries<D, 16, 2, INTER>(p, at, turns);
    else append_queries<D, 4, 2, INTER>(p, at, turns);
    return;
  }
  at -= g.q_blocks;
  append_page<D>(p.a, 1, (int)(at % (unsigned)p.a.p.heads), (int)(at / (unsigned)p.a.p.heads));
}

// One token of every sequence: a warp per sequence, head and K or V, half the lanes
// a unit of 16 channels each; behind them blocks of query rows.  What counts is
// the chain of dependent loads: length, position, then turns beside table entry
// and scale.
constexpr int kOneRows = 4;   // append_query_rows
template <int D, bool INTER>
__global__ void __launch_bounds__(128) append_one_rope_kernel(const __grid_constant__ AppendRopeArgs p, unsigned kv_blocks) {
  constexpr int U = D / 16;
  __shared__ float4 turns[kOneRows * kRopeRow];   // of the block's four warps, or its query rows
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  if (blockIdx.x >= kv_blocks) {
    append_queries<D, kOneRows, 2, INTER>(p, blockIdx.x - kv_blocks, turns);
    return;
  }
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int kv = (int)(w & 1), head = (int)((w >> 1) % a.p.heads);
  const long long item = (w >> 1) / a.p.heads;
  if (item >= a.s.batch) return;
  const int b = (int)item;
  const bool has = lane < U;
  int c0, c1;
  rope_chunks(p.t, lane % U, c0, c1);
  uint4 v = make_uint4(0u, 0u, 0u, 0u), y = v;
  if (has) {
    const uint16_t* from = a.x[kv] + b * a.row_stride[kv] + head * a.head_stride[kv];
    v = __ldg(reinterpret_cast<const uint4*>(from + c0));
    y = __ldg(reinterpret_cast<const uint4*>(from + c1));
  }
  const int len = seq_len(a.s, b, a.p.shift, a.status);
  if (len < 1) {
    page_error(a.status);     // a new token, but no place for it
    return;
  }
  const int pg = (len - 1) >> a.p.shift, t = (len - 1) & (a.p.page - 1);
  float f[8], g[8];
  floats_of(v, f);
  floats_of(y, g);
  if (kv == 0) {   // the warp's own row of turns
    float4* row = turns + (threadIdx.x >> 5) * kRopeRow;
    rope_stage_one(p.t, row, a.status, a.bounds_site, [&](int axis) { return p.pos != nullptr ? __ldg(p.pos + b * p.pr + axis) : len - 1; });
    __syncwarp();
    if (lane < (p.t.pairs >> 3)) {
      float4 cs[4];
      rope_entries(row, lane, cs);
      rope_apply<INTER>(p.t, cs, v, y, f, g);
    }
  }
  const int id = seq_page(a.s, b, pg, a.p.n_pages, a.status);
  if (id < 0) return;
  const long long blk = (long long)id * a.p.heads + head;
  if (!KVQ_IN_BOUNDS(blk, (long long)a.p.n_pages * a.p.heads, a.status, a.bounds_site)) return;
  uint8_t* codes = a.p.codes[kv] + blk * a.p.page * D;
  const int old = t > 0 ? scale_exp(a.p.scale[kv][blk]) : kPageExpMin;
  const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(most_of(0.f, f, g)));
  const int e = max(scale_of(__uint_as_float(m), a.status), old);
  if (t > 0 && e > old) rescale_codes<D>(codes, t, old - e, lane, 32);
  if (lane == 0 && (t == 0 || e > old)) a.p.scale[kv][blk] = scale_bits(e);
  if (has) {
    *reinterpret_cast<uint2*>(codes + t * D + c0) = codes_of(f, pow2f(-e));
    *reinterpret_cast<uint2*>(codes + t * D + c1) = codes_of(g, pow2f(-e));
  }
}

std::atomic<uint64_t> g_append_smem[2][2];

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
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  auto blocks = [&](int tile) {
    return a.batch * (rope_blocks(a.rows, a.x[0].heads, tile) + rope_blocks(a.rows, a.x[1].heads, tile));
  };
  // few rows: four a block, as long as those do not fill the GPU twice
  const bool few = blocks(4) <= 16LL * sms;
  auto pick = [&](auto inter) {
    constexpr bool I = decltype(inter)::value;
    return few ? (a.d == 64 ? rope_kernel<64, 4, I> : rope_kernel<128, 4, I>)
               : (a.d == 64 ? rope_kernel<64, 16, I> : rope_kernel<128, 16, I>);
  };
  const auto kern = a.t.interleaved ? pick(std::true_type{}) : pick(std::false_type{});
  return launch_dependent(kern, (unsigned)blocks(few ? 4 : 16), 256, 0, stream, a);
}

cudaError_t launch_pages_append_rope(const AppendRopeArgs& p, cudaStream_t stream) {
  const AppendArgs& a = p.a;
  const int sms = sm_count_current();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int q_rows = append_query_rows(a.s.offsets == nullptr, a.p.page);
  const long long q_blocks = rope_blocks(a.s.rows, p.q.heads, q_rows);
  if (a.s.offsets == nullptr) {
    const long long kv_blocks = ((long long)a.s.batch * a.p.heads * 2 + 3) / 4;
    auto pick = [&](auto inter) {
      constexpr bool I = decltype(inter)::value;
      return a.p.d == 64 ? append_one_rope_kernel<64, I> : append_one_rope_kernel<128, I>;
    };
    const auto kern = p.t.interleaved ? pick(std::true_type{}) : pick(std::false_type{});
    return launch_dependent(kern, (unsigned)(kv_blocks + q_blocks), 128, 0, stream, p, (unsigned)kv_blocks);
  }
  const long long items = append_items(a.s.rows, a.s.batch, a.p.shift);
  AppendGrid g{};
  g.heads = 8;   // a block of keys, as long as there is one for every SM
  while (g.heads > 1 && items * ((a.p.heads + g.heads - 1) / g.heads) < sms) g.heads /= 2;
  g.k_blocks = (unsigned)(items * ((a.p.heads + g.heads - 1) / g.heads));
  g.q_rows = q_rows;
  g.q_blocks = (unsigned)q_blocks;
  const unsigned v_blocks = (unsigned)(items * a.p.heads);
  const int smem = a.p.page * kRopeRow * (int)sizeof(float4);
  auto pick = [&](auto inter) {
    constexpr bool I = decltype(inter)::value;
    return a.p.d == 64 ? append_rope_kernel<64, I> : append_rope_kernel<128, I>;
  };
  const auto kern = p.t.interleaved ? pick(std::true_type{}) : pick(std::false_type{});
  const cudaError_t e = ensure_smem_limit(kern, 128 * kRopeRow * (int)sizeof(float4), g_append_smem[a.p.d == 128][p.t.interleaved]);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, g.k_blocks + g.q_blocks + v_blocks, a.p.page * a.p.d / 32, smem, stream, p, g);
}

}  // namespace kvq
