// Attention over the paged 8-bit cache (sm_103a): plain scores, and what the
// modes of the kernels share.
#include "kvq_paged_launch.cuh"

namespace kvq {
namespace {

// Clusters of c = 2^k CTAs of the item kernel that run at once on the current
// device (its SMs come in groups that a cluster cannot straddle: of 152 SMs 76
// clusters of 2, 36 of 4, 15 of 8, 7 of 16); asked once per device.
int active_clusters(int k) {
  static std::atomic<int> known[64][5];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int had = known[dev][k].load(std::memory_order_relaxed);
  if (had != 0) return had - 1;
  const auto kern = decode_item_kernel<128, 1, kDecWarps, kPlain>;
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
  if (ensure_smem_limit(kern, smem, (DecodeOnce<128, 1, kDecWarps, kPlain>::item)) != cudaSuccess ||
      ensure_wide_clusters(kern, (DecodeOnce<128, 1, kDecWarps, kPlain>::wide)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();   // no clusters, then
    n = 0;
  }
  known[dev][k].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

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
  return launch_paged_mode<kPlain>(a, stream);
}

kvq_status launch_paged_attention_scored(const PagedAttnArgs& a, cudaStream_t stream) {
  return a.shape.cap > 0.f ? launch_paged_capped(a, stream) : launch_paged_biased(a, stream);
}

}  // namespace kvq
