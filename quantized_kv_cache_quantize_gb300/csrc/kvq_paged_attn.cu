// Attention over the paged 8-bit cache (sm_103a).
#include <cuda_runtime.h>

#include <math_constants.h>

#include <algorithm>

#include "kvq_checks.cuh"
#include "kvq_paged_chunk.cuh"
#include "kvq_paged_decode.cuh"
#include "kvq_pages.cuh"
#include "kvq_tmap.cuh"

namespace kvq {
namespace {

// ---- few rows: the decoding form ----
// Rows of a cache head up to which the decoding form is taken: two column
// tiles are what a warp's registers hold.  Past them it would read the keys
// again from L2, and the tensor-core form, which works on 128 rows however few
// there are, is as good or better.  Decoding / tensor-core form in us, 32
// sequences of 16384 keys, 8 heads of 128 channels: 16 rows 186 / 258, 24 rows
// (in two passes, measured before the present form) 343 / 258; 64 channels:
// 145 / 222, 278 / 222.
constexpr int kDecRows = 16;

std::atomic<uint64_t> g_decode_smem[2][2], g_decode12_smem[2], g_item_smem[2][2], g_item_wide[2][2];

// clusters of more than 8 CTAs, allowed once per kernel and device
template <typename Kernel>
cudaError_t ensure_wide_clusters(Kernel kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t{1} << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Warps of the decoding form, per CTA.  Twelve hide more of the latency of
// products and votes than eight where every warp has a long run of keys
// (94 against 110 us: 32 sequences of 16384 keys, 8 heads of 64 channels);
// with short runs the larger CTA's start costs more (20.5 against 17.8 us: 16
// of 4096, 4 heads of 128).  Two column tiles have no registers for twelve.
constexpr int kDecWarps = 8, kDecWarpsLong = 12, kLongUnits = 16;
int decode_warps(int sms, int row_tiles, double units) {
  return row_tiles == 1 && units >= (double)kLongUnits * kDecWarps * sms ? kDecWarpsLong : kDecWarps;
}
double decode_units(long long items, long long keys) { return (double)items * ((double)keys / kUnit + 1.0); }

struct DecodeWs {
  size_t ml, o, bytes;   // the first units come first
};
DecodeWs decode_ws(int warps, int batch, int rows_cap, int d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t slots = 2 * (size_t)warps * rows_cap;
  DecodeWs w{};
  w.ml = up(((size_t)batch + 1) * 8);
  w.o = w.ml + up(slots * 8);
  w.bytes = w.o + up(slots * d * 4);
  return w;
}

// Clusters of c = 2^k CTAs of the item kernel that run at once on the current
// device (its SMs come in groups that a cluster cannot straddle: of 152 SMs 76
// clusters of 2, 36 of 4, 15 of 8, 7 of 16); asked once per device.
int active_clusters(int k) {
  static std::atomic<int> known[64][5];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int had = known[dev][k].load(std::memory_order_relaxed);
  if (had != 0) return had - 1;
  const auto kern = decode_item_kernel<128, 1, kDecWarps>;
  const int smem = DecCfg<128, kDecWarps>::kAlloc;
  int n = 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(64u << k);
  cfg.blockDim = dim3(kDecWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1u << k;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (ensure_smem_limit(kern, smem, g_item_smem[1][0]) != cudaSuccess ||
      ensure_wide_clusters(kern, g_item_wide[1][0]) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();   // no clusters, then
    n = 0;
  }
  known[dev][k].store(n + 1, std::memory_order_relaxed);
  return n;
}

// CTAs per item (sequence, cache head, row group), or 0 for equal runs of the
// line of all keys.  An item's CTAs start at once and join by themselves, but
// the longest item decides; the line scans the batch, takes a second kernel,
// which joins every item's pieces, and balances.  The times below, in us, are
// fits to measured ones (sequences of one length; 128 channels, grouped by 4,
// item / line): 32 items of 512 keys 6.7 / 10.0, of 8192 15.8 / 18.7; 64 of
// 8192 26.7 / 33.3; 48 of 32768 78.8 / 75.9; 192 of 2048 27.5 / 24.3; 4 of 32768
// 16.6 / 23.1.  Keys are known by the table's width only, so a CTA's share is limited
// too, to 4096 keys: the longest of a ragged batch then costs 25 us at most.
int decode_by_item(int sms, int d, long long items, long long keys) {
  if (items > 2LL * sms) return 0;
  int c = 1;
  for (int k = 1; (1 << k) <= kMaxCluster && items <= active_clusters(k); ++k) c = 1 << k;
  const double units = (double)keys / kUnit, share = (double)((items + sms - 1) / sms) * units / c;
  if (share > 128.0) return 0;
  const double unit = d == 128 ? 0.16 : 0.12;
  const double t_item = (c > 1 || items > sms ? 5.5 : 3.8) + unit * share;
  const double pieces = std::min(units, (double)sms * kDecWarps / (double)items);
  const double t_line = 8.7 + 0.02 * pieces + 1.25 * unit * units * (double)items / sms;
  return t_item < t_line ? c : 0;
}

// Keys of a sequence that its rows attend to, at most: the table's width, or
// the window's keys before its last max_q tokens.  (Fewer keys never need more
// workspace: the size asked for is that of the width.)
long long key_bound(const PagedAttnArgs& a) {
  const long long keys = (long long)a.s.width * a.p.page;
  return a.window > 0 ? std::min(keys, (long long)a.window + a.max_q) : keys;
}

template <int D, int NT>
kvq_status launch_decode(const PagedAttnArgs& a, cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int cap = a.max_q * a.group;
  const long long items = (long long)a.s.batch * a.p.heads;
  CUtensorMap mk, mv;
  const long long blocks = (long long)a.p.n_pages * a.p.heads;
  const int box = a.p.page < kUnit ? a.p.page : kUnit;
  if (!make_pages_map(&mk, a.p.codes[0], D, a.p.page, blocks, box) ||
      !make_pages_map(&mv, a.p.codes[1], D, a.p.page, blocks, box))
    return KVQ_ERR_CUDA;
  const int smem = DecCfg<D, kDecWarps>::kAlloc;
  DecodeArgs d{};
  d.a = a;
  d.rows_cap = cap;
  d.cluster = decode_by_item(sms, D, items, key_bound(a));
  if (d.cluster > 0) {
    const auto kern = decode_item_kernel<D, NT, kDecWarps>;
    if (ensure_smem_limit(kern, smem, g_item_smem[D == 128][NT - 1]) != cudaSuccess ||
        (d.cluster > 8 && ensure_wide_clusters(kern, g_item_wide[D == 128][NT - 1]) != cudaSuccess) ||
        launch_clusters(kern, (unsigned)(items * d.cluster), (unsigned)d.cluster, kDecWarps * 32, smem, stream, d, mk,
                        mv) != cudaSuccess)
      return KVQ_ERR_CUDA;
    return KVQ_OK;
  }
  // the units there can be bound the grid
  const double most = decode_units(items, key_bound(a));
  const int warps = decode_warps(sms, NT, most);
  const DecodeWs ws = decode_ws(sms * warps, a.s.batch, cap, D);
  if (a.ws_bytes < ws.bytes) return KVQ_ERR_INVALID_ARG;
  int grid = sms;
  if (most < (double)sms * warps * kMinUnits) grid = std::min((int)(most / kMinUnits) + 1, sms);
  uint8_t* base = static_cast<uint8_t*>(a.ws);
  d.pre = reinterpret_cast<long long*>(base);
  d.part_ml = reinterpret_cast<float*>(base + ws.ml);
  d.part_o = reinterpret_cast<float*>(base + ws.o);
  d.warps = grid * warps;
  if constexpr (NT == 1) {
    if (warps == kDecWarpsLong) {
      const auto kern = decode_kernel<D, NT, kDecWarpsLong>;
      const int bytes = DecCfg<D, kDecWarpsLong>::kAlloc;
      if (ensure_smem_limit(kern, bytes, g_decode12_smem[D == 128]) != cudaSuccess ||
          launch_dependent(kern, (unsigned)grid, kDecWarpsLong * 32, bytes, stream, d, mk, mv) != cudaSuccess)
        return KVQ_ERR_CUDA;
    }
  }
  if (warps == kDecWarps) {
    const auto kern = decode_kernel<D, NT, kDecWarps>;
    if (ensure_smem_limit(kern, smem, g_decode_smem[D == 128][NT - 1]) != cudaSuccess ||
        launch_dependent(kern, (unsigned)grid, kDecWarps * 32, smem, stream, d, mk, mv) != cudaSuccess)
      return KVQ_ERR_CUDA;
  }
  const long long rows = (long long)a.s.batch * a.p.heads * cap;
  if (launch_dependent(join_kernel<D>, (unsigned)rows, kJoinWarps * 32, 0, stream, d) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}

// ---- many rows: the tensor-core form ----
std::atomic<uint64_t> g_chunk_smem[2][2];
constexpr int kMaxSplits = 32;

// Key ranges per row tile at most: what fills the SMs twice over.
int split_limit(int sms, long long ctas) {
  const long long s = ctas > 0 ? (2LL * sms + ctas - 1) / ctas : 1;
  return (int)(s > kMaxSplits ? kMaxSplits : s);
}
// Query tiles of 128 rows a CTA: one or two.  Two against one in us, 32
// sequences of 16384 keys, 8 heads of 128 channels: 128 rows 418 / 267, 144
// rows 438 / 518, 256 rows 447 / 530; 16 of 4096: 61.6 / 43.6, 64.9 / 81.3,
// 67.8 / 83.9.  (With few CTAs, 4 sequences of 2048 keys, one is the better at
// 256 rows, 28.0 / 24.8, and past that.)
int query_tiles(long long cap) { return cap <= 128 ? 1 : 2; }
long long chunk_tiles(int batch, int heads, long long cap, int* q_tiles) {
  const int per = 128 * query_tiles(cap);
  *q_tiles = (int)((cap + per - 1) / per);
  return (long long)batch * heads * *q_tiles;
}
size_t chunk_ws(int splits, int rows, int q_heads, int d) {
  return splits > 1 ? (size_t)splits * rows * q_heads * (d + 2) * 4 + 16 : 16;
}

template <int D, int NQ>
kvq_status launch_chunk(const PagedAttnArgs& a, cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return KVQ_ERR_CUDA;
  ChunkArgs c{};
  c.a = a;
  const long long cap = (long long)a.max_q * a.group;
  const long long ctas = chunk_tiles(a.s.batch, a.p.heads, cap, &c.q_tiles);
  // ranges: the cost model of the window attention's key-range split
  int max_splits = split_limit(sms, ctas), per = 0;
  while (max_splits > 1 && chunk_ws(max_splits, a.s.rows, a.q_heads, D) > a.ws_bytes) --max_splits;
  const long long keys = key_bound(a);
  attention_split((long long)a.s.batch * a.p.heads, (int)cap, (int)((keys + 127) / 128), 0, D, 128 * NQ, sms,
                  max_splits, &c.splits, &per);
  if (a.ws_bytes < chunk_ws(c.splits, a.s.rows, a.q_heads, D)) return KVQ_ERR_INVALID_ARG;
  c.part_o = static_cast<float*>(a.ws);
  c.part_ml = c.part_o + (size_t)c.splits * a.s.rows * a.q_heads * D;
  if (ctas * c.splits > 0x7fffffffLL) return KVQ_ERR_TOO_LARGE;
  CUtensorMap mk, mv;
  const long long blocks = (long long)a.p.n_pages * a.p.heads;
  if (!make_pages_map(&mk, a.p.codes[0], D, a.p.page, blocks, a.p.page) ||
      !make_pages_map(&mv, a.p.codes[1], D, a.p.page, blocks, a.p.page))
    return KVQ_ERR_CUDA;
  using Cfg = ChunkCfg<D, NQ>;
  if (ensure_smem_limit(chunk_kernel<D, NQ>, Cfg::kAlloc, g_chunk_smem[D == 128][NQ - 1]) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (launch_dependent(chunk_kernel<D, NQ>, (unsigned)(ctas * c.splits), Cfg::kThreads, Cfg::kAlloc, stream, c, mk,
                       mv) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (c.splits > 1) {
    const long long warps = (long long)a.s.batch * a.max_q * a.q_heads;
    if ((warps + 7) / 8 > 0x7fffffffLL) return KVQ_ERR_TOO_LARGE;
    if (launch_dependent(chunk_join_kernel<D>, (unsigned)((warps + 7) / 8), 256, 0, stream, c) != cudaSuccess)
      return KVQ_ERR_CUDA;
  }
  return KVQ_OK;
}

}  // namespace

size_t paged_attention_workspace(int kv_heads, int q_heads, int d, int batch, long long keys, int rows, int max_q) {
  if (max_q > rows) max_q = rows;
  const long long cap = (long long)max_q * (q_heads / kv_heads);
  const int sms = std::max(sm_count_current(), 1);
  if (cap <= kDecRows) {
    const long long items = (long long)batch * kv_heads;
    if (decode_by_item(sms, d, items, keys) > 0) return 16;
    return decode_ws(sms * decode_warps(sms, cap <= 8 ? 1 : 2, decode_units(items, keys)), batch, (int)cap, d).bytes;
  }
  int q_tiles = 0;
  return chunk_ws(split_limit(sms, chunk_tiles(batch, kv_heads, cap, &q_tiles)), rows, q_heads, d);
}

kvq_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream) {
  const long long cap = (long long)a.max_q * a.group;
  if (cap > 0x3fffffffLL || (long long)a.s.batch * a.p.heads > 0x7fffffffLL / (cap <= kDecRows ? kDecRows : 1))
    return KVQ_ERR_TOO_LARGE;
  if (cap <= kDecRows) {
    if (a.p.d == 64) return cap > 8 ? launch_decode<64, 2>(a, stream) : launch_decode<64, 1>(a, stream);
    return cap > 8 ? launch_decode<128, 2>(a, stream) : launch_decode<128, 1>(a, stream);
  }
  if (a.p.d == 64) return query_tiles(cap) == 2 ? launch_chunk<64, 2>(a, stream) : launch_chunk<64, 1>(a, stream);
  return query_tiles(cap) == 2 ? launch_chunk<128, 2>(a, stream) : launch_chunk<128, 1>(a, stream);
}

}  // namespace kvq
