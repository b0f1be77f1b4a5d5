// Attention over the paged 8-bit cache (sm_103a).
#include <cuda_runtime.h>

#include <math_constants.h>

#include <algorithm>

#include "kvq_checks.cuh"
#include "kvq_paged_decode.cuh"
#include "kvq_pages.cuh"
#include "kvq_tmap.cuh"

namespace kvq {
namespace {

// One warp per query row and head; every lane holds D / 32 channels.
template <int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int qh = (int)(w % a.q_heads);
  const long long rb = w / a.q_heads;
  const int i = (int)(rb % a.max_q), b = (int)(rb / a.max_q);
  if (b >= a.s.batch) return;
  int r0, n;
  seq_rows(a.s, b, r0, n, a.status);
  if (n > a.max_q) page_error(a.status);
  if (i >= n) return;
  const int len = seq_len(a.s, b, a.p.shift, a.status);
  const int t = len - n + i, head = qh / a.group;
  const int hi = a.causal ? min(len, t + 1) : len;
  const int lo = a.window > 0 ? max(0, t - a.window + 1) : 0;
  const long long row = r0 + i;
  float q[C], o[C];
  for (int c = 0; c < C; ++c) {
    q[c] = a.scale * __uint_as_float((uint32_t)a.q[row * a.q_row_stride + qh * a.q_head_stride + C * lane + c] << 16);
    o[c] = 0.f;
  }
  float top = -CUDART_INF_F, sum = 0.f;
  int id = -1;
  float ks = 0.f, vs = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int in = j & (a.p.page - 1);
    if (in == 0 || j == lo) {
      id = seq_page(a.s, b, j >> a.p.shift, a.p.n_pages, a.status);
      if (id >= 0) {
        ks = pow2f(scale_exp(a.p.scale[0][(long long)id * a.p.heads + head]));
        vs = pow2f(scale_exp(a.p.scale[1][(long long)id * a.p.heads + head]));
      }
    }
    if (id < 0) continue;
    const long long at = (((long long)id * a.p.heads + head) * a.p.page + in) * D + C * lane;
    float s = 0.f;
    float v[C];
    for (int c = 0; c < C; c += 2) {
      const uint32_t kh = f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t*>(a.p.codes[0] + at + c));
      const uint32_t vh = f16x2_of_e4m3x2(*reinterpret_cast<const uint16_t*>(a.p.codes[1] + at + c));
      const float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(&kh));
      const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&vh));
      s += q[c] * k2.x + q[c + 1] * k2.y;
      v[c] = v2.x * vs;
      v[c + 1] = v2.y * vs;
    }
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= ks;
    const float next = fmaxf(top, s);
    const float f = expf(top - next), e = expf(s - next);
    sum = sum * f + e;
    for (int c = 0; c < C; ++c) o[c] = o[c] * f + e * v[c];
    top = next;
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  for (int c = 0; c < C; ++c) {
    const __nv_bfloat16 v = __float2bfloat16_rn(o[c] * inv);
    a.out[(row * a.q_heads + qh) * D + C * lane + c] = *reinterpret_cast<const uint16_t*>(&v);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[row * a.q_heads + qh] = sum > 0.f ? top + logf(sum) : -CUDART_INF_F;
}

// ---- few rows: the decoding form ----
constexpr int kDecRows = 16;

std::atomic<uint64_t> g_decode_smem[2][2];

template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), unsigned grid, int threads, int smem,
                             cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct DecodeWs {
  size_t pre, ml, o, bytes;
};
DecodeWs decode_ws(int sms, int batch, int rows_cap, int d) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t slots = 2 * (size_t)sms * kDecWarps * rows_cap;
  DecodeWs w{};
  w.ml = up(((size_t)batch + 1) * 8);
  w.o = w.ml + up(slots * 8);
  w.bytes = w.o + up(slots * d * 4);
  return w;
}

template <int D, int NT>
kvq_status launch_decode(const PagedAttnArgs& a, cudaStream_t stream) {
  const int sms = sm_count_current();
  if (sms <= 0) return KVQ_ERR_CUDA;
  const int rows_cap = a.max_q * a.group;
  const DecodeWs ws = decode_ws(sms, a.s.batch, rows_cap, D);
  if (a.ws_bytes < ws.bytes) return KVQ_ERR_INVALID_ARG;
  // the units there can be, from the table's width, bound the grid
  const double most = (double)a.s.batch * a.p.heads * ((double)a.s.width * a.p.page / kUnit + 1.0);
  int grid = sms;
  if (most < (double)sms * kDecWarps * kMinUnits) {
    grid = (int)(most / kMinUnits) + 1;
    if (grid > sms) grid = sms;
  }
  DecodeArgs d{};
  d.a = a;
  uint8_t* base = static_cast<uint8_t*>(a.ws);
  d.pre = reinterpret_cast<long long*>(base + ws.pre);
  d.part_ml = reinterpret_cast<float*>(base + ws.ml);
  d.part_o = reinterpret_cast<float*>(base + ws.o);
  d.rows_cap = rows_cap;
  d.warps = grid * kDecWarps;
  CUtensorMap mk, mv;
  const long long blocks = (long long)a.p.n_pages * a.p.heads;
  const int box = a.p.page < kUnit ? a.p.page : kUnit;
  if (!make_pages_map(&mk, a.p.codes[0], D, a.p.page, blocks, box) ||
      !make_pages_map(&mv, a.p.codes[1], D, a.p.page, blocks, box))
    return KVQ_ERR_CUDA;
  const int smem = DecCfg<D>::kAlloc;
  if (ensure_smem_limit(decode_kernel<D, NT>, smem, g_decode_smem[D == 128][NT - 1]) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (launch_dependent(decode_kernel<D, NT>, (unsigned)grid, kDecWarps * 32, smem, stream, d, mk, mv) !=
      cudaSuccess)
    return KVQ_ERR_CUDA;
  const long long items = (long long)a.s.batch * a.p.heads;
  if (launch_dependent(join_kernel<D>, (unsigned)items, kJoinWarps * 32, 0, stream, d) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}

}  // namespace

size_t paged_attention_workspace(int kv_heads, int q_heads, int d, int batch, int rows, int max_q) {
  if (max_q > rows) max_q = rows;
  const long long cap = (long long)max_q * (q_heads / kv_heads);
  if (cap > kDecRows) return 16;
  return decode_ws(std::max(sm_count_current(), 1), batch, (int)cap, d).bytes;
}

kvq_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream) {
  const long long items = (long long)a.s.batch * a.p.heads;
  if ((long long)a.max_q * a.group <= kDecRows && items <= 0x7fffffffLL) {
    const bool wide = a.max_q * a.group > 8;
    if (a.p.d == 64) return wide ? launch_decode<64, 2>(a, stream) : launch_decode<64, 1>(a, stream);
    return wide ? launch_decode<128, 2>(a, stream) : launch_decode<128, 1>(a, stream);
  }
  const long long warps = (long long)a.s.batch * a.max_q * a.q_heads;
  const long long grid = (warps + 3) / 4;
  if (grid > 0x7fffffffLL) return KVQ_ERR_TOO_LARGE;
  if (a.p.d == 64) paged_attn_kernel<64><<<(unsigned)grid, 128, 0, stream>>>(a);
  else paged_attn_kernel<128><<<(unsigned)grid, 128, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
