// Attention over the paged cache with shaped scores (sm_103a).
#include <cuda_runtime.h>

#include <math_constants.h>

#include "kvq_checks.cuh"
#include "kvq_scores.cuh"

namespace kvq {
namespace {

// A warp per query row and head: 32 keys at a time, a key a lane for the
// scores, d / 32 channels a lane for the output.
template <int D>
__global__ void __launch_bounds__(128) scored_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int C = D / 32;
  __shared__ float qs[4][D];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  ptx::grid_dependency_wait();
  const long long w = (long long)blockIdx.x * 4 + wid;
  const int hq = (int)(w % a.q_heads);
  const long long rb = w / a.q_heads;
  const int i = (int)(rb % a.max_q);
  const long long bl = rb / a.max_q;
  if (bl >= a.s.batch) return;
  const int b = (int)bl, h = hq / a.group;
  int r0, n;
  seq_rows(a.s, b, r0, n, a.status);
  if (n > a.max_q) {
    page_error(a.status);
    n = a.max_q;
  }
  if (i >= n) return;
  const int len = seq_len(a.s, b, a.p.shift, a.status);
  const RowView v = row_view(a, b, r0 + i, len - n + i, len);
  const uint16_t* qp = a.q + (long long)(r0 + i) * a.q_row_stride + (long long)hq * a.q_head_stride;
  bool fine = true;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float x = __uint_as_float((uint32_t)qp[lane + 32 * c] << 16);
    fine = fine && fabsf(x) < CUDART_INF_F;
    qs[wid][lane + 32 * c] = x;
  }
  if (!__all_sync(0xffffffffu, fine))   // an infinity or a NaN makes the whole row NaN
    for (int c = 0; c < C; ++c) qs[wid][lane + 32 * c] = CUDART_NAN_F;
  __syncwarp();
  const float cap = a.shape.cap, slope = a.shape.slopes != nullptr ? __ldg(a.shape.slopes + hq) : 0.f;
  float m = -CUDART_INF_F, l = 0.f, o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  for (int j0 = v.lo & ~15; j0 < v.hi; j0 += 32) {
    const int j = j0 + lane;
    int id = -1;
    if (j >= v.lo && j < v.hi) id = seq_page(a.s, b, j >> a.p.shift, a.p.n_pages, a.status);
    const long long blk = (long long)id * a.p.heads + h, at = (blk << a.p.shift) + (j & (a.p.page - 1));
    float s = -CUDART_INF_F, fv = 0.f;
    if (id >= 0) {
      const uint4* k = reinterpret_cast<const uint4*>(a.p.codes[0] + at * D);
      float acc = 0.f;
      for (int c = 0; c < D / 16; ++c) {
        const uint4 x = __ldg(k + c);
        const uint32_t word[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t p = f16x2_of_e4m3x2((uint16_t)(word[u >> 1] >> (16 * (u & 1))));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
          acc = fmaf(f.x, qs[wid][16 * c + 2 * u], acc);
          acc = fmaf(f.y, qs[wid][16 * c + 2 * u + 1], acc);
        }
      }
      s = acc * a.scale * pow2f(scale_exp(__ldg(a.p.scale[0] + blk)));
      if (cap > 0.f) s = cap * tanhf(s / cap);
      s = fmaf(-slope, (float)abs(v.ref - j), s);
      fv = pow2f(scale_exp(__ldg(a.p.scale[1] + blk)));
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float mn = fmaxf(m, top), base = mn > -CUDART_INF_F ? mn : 0.f;
    const float p = expf(s - base), down = expf(m - base);
    m = mn;
    l *= down;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] *= down;
    l += p;   // this lane's keys
    for (int u = 0; u < 32; ++u) {
      const float pu = __shfl_sync(0xffffffffu, p, u), f = __shfl_sync(0xffffffffu, fv, u);
      const long long au = __shfl_sync(0xffffffffu, at, u);
      if (f == 0.f) continue;
      const uint8_t* x = a.p.codes[1] + au * D + C * lane;
#pragma unroll
      for (int c = 0; c < C; c += 2) {
        const uint32_t y = f16x2_of_e4m3x2(__ldg(reinterpret_cast<const uint16_t*>(x + c)));
        const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&y));
        o[c] = fmaf(pu, z.x * f, o[c]);
        o[c + 1] = fmaf(pu, z.y * f, o[c + 1]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const long long row = (long long)(r0 + i) * a.q_heads + hq;
  if (!KVQ_IN_BOUNDS(row, (long long)a.s.rows * a.q_heads, a.status, a.bounds_site)) return;
  const float f = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < C; c += 2) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(o[c] * f, o[c + 1] * f);
    *reinterpret_cast<uint32_t*>(a.out + row * D + C * lane + c) = *reinterpret_cast<const uint32_t*>(&z);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -CUDART_INF_F : m + logf(l) + ref_bias(a, v, hq);
}

}  // namespace

kvq_status launch_paged_attention_scored(const PagedAttnArgs& a, cudaStream_t stream) {
  const long long warps = (long long)a.s.batch * a.max_q * a.q_heads;
  if ((warps + 3) / 4 > 0x7fffffffLL) return KVQ_ERR_TOO_LARGE;
  const auto kern = a.p.d == 64 ? scored_kernel<64> : scored_kernel<128>;
  return launch_dependent(kern, (unsigned)((warps + 3) / 4), 128, 0, stream, a) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
