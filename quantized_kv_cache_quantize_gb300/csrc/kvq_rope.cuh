// Device helpers of the rotary positions: rows' positions, cosines and sines
// from the table, the rotation itself.
#pragma once

#include "kvq_pages.cuh"

namespace kvq {
namespace {

// a row's position, held inside the table (one outside it is recorded)
__device__ __forceinline__ int rope_position(const RopeTab& t, int p, int* status) {
  if ((unsigned)p >= (unsigned)t.n) {
    atomicCAS(status, 0, (int)KVQ_ERR_POSITION);
    p = min(max(p, 0), t.n - 1);
  }
  return p;
}

// Turns of rows in shared memory, kRopeRow entries (the cosines, then the sines of
// two pairs) a row: entry e, of pairs 2 e and 2 e + 1, stands where lanes that
// write neighbouring entries, and lanes that read the same entry of neighbouring
// units (of 8 pairs), meet different banks.
constexpr int kRopeRow = kRopeMaxPairs / 2;
__device__ __forceinline__ int rope_slot(int unit, int j) { return 8 * j + (unit ^ (2 * j)); }
// A row's, by a warp, a lane an entry.  pos(axis): the row's position.
template <typename Pos>
__device__ __forceinline__ void rope_stage_one(const RopeTab& t, float4* row, int* status, Pos pos, bool inverse = false) {
  const int e = threadIdx.x & 31, p = 2 * e;
  if (p >= t.pairs) return;
  const int axis0 = t.axis[p], axis1 = t.axis[p + 1];
  const float2* from = t.cs + (long long)rope_position(t, pos(axis0), status) * t.pairs + p;
  float4 v;   // cos, sin, cos, sin
  if (axis0 == axis1) {
    v = __ldg(reinterpret_cast<const float4*>(from));
  } else {
    const float2 x = __ldg(from), y = __ldg(t.cs + (long long)rope_position(t, pos(axis1), status) * t.pairs + p + 1);
    v = make_float4(x.x, x.y, y.x, y.y);
  }
  row[rope_slot(e >> 2, e & 3)] = inverse ? make_float4(v.x, v.z, -v.y, -v.w) : make_float4(v.x, v.z, v.y, v.w);
}
// Those of `rows` rows by a block, a warp a row.  pos(row, axis): a row's position.
template <typename Pos>
__device__ __forceinline__ void rope_stage(const RopeTab& t, float4* turns, int rows, bool inverse, int* status, Pos pos) {
  for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5)
    rope_stage_one(t, turns + r * kRopeRow, status, [&](int axis) { return pos(r, axis); }, inverse);
}

__device__ __forceinline__ void floats_of(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 bf16_of(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&z);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two pairs: x0, x1 their first and second channels.  Each product and sum is
// rounded by itself: the bits are those of the formula evaluated step by step in
// fp32, whatever else a kernel does around it.  (Products on pairs would be fused
// with the sums behind them, and rounded once.)
__device__ __forceinline__ void turn_pairs(float (&x0)[2], float (&x1)[2], const float4& cs) {
  const float c[2] = {cs.x, cs.y}, s[2] = {cs.z, cs.w};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = x0[i], b = x1[i];
    x0[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
    x1[i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
  }
}

// 16 channels of a row, unit u of d / 16: where u < pairs / 8, the channels of
// pairs [8 u, 8 u + 8) in two 16-byte chunks, rotated; behind them 16 channels
// that stay.  `c0`, `c1`: the chunks, in elements.
__device__ __forceinline__ void rope_chunks(const RopeTab& t, int u, int& c0, int& c1) {
  const bool halves = u < (t.pairs >> 3) && !t.interleaved;
  c0 = halves ? 8 * u : 16 * u;
  c1 = halves ? c0 + t.pairs : c0 + 8;
}
// The unit's chunks a, b as fp32 f, g, rotated by the row's turns.
__device__ __forceinline__ void rope_apply(const RopeTab& t, const float4* row, int u, const uint4& a, const uint4& b,
                                           float (&f)[8], float (&g)[8]) {
  floats_of(a, f);
  floats_of(b, g);
  if (t.interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float(&z)[8] = j < 2 ? f : g;
      const int k = 4 * (j & 1);
      float x0[2] = {z[k], z[k + 2]}, x1[2] = {z[k + 1], z[k + 3]};
      turn_pairs(x0, x1, row[rope_slot(u, j)]);
      z[k] = x0[0], z[k + 2] = x0[1], z[k + 1] = x1[0], z[k + 3] = x1[1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x0[2] = {f[2 * j], f[2 * j + 1]}, x1[2] = {g[2 * j], g[2 * j + 1]};
      turn_pairs(x0, x1, row[rope_slot(u, j)]);
      f[2 * j] = x0[0], f[2 * j + 1] = x0[1], g[2 * j] = x1[0], g[2 * j + 1] = x1[1];
    }
  }
}

// R rows of up to kRopeHeads heads of one tensor by a block: the values are asked
// for first, then the rows' turns go through shared memory (R * kRopeRow), read
// once for all heads.  x, y: row 0, head 0.
constexpr int kRopeHeads = 8;
template <int D, int R, typename Pos>
__device__ __forceinline__ void rope_tile(const RopeTab& t, bool inverse, float4* turns, int rows, int heads,
                                          const uint16_t* x, long long xr, long long xh, uint16_t* y, long long yr,
                                          long long yh, int* status, Pos pos) {
  constexpr int U = D / 16, kAll = R * kRopeHeads * U, N = R >= 16 ? 4 : 1;
  const int step = (int)blockDim.x;
  bool staged = false;
  for (int i0 = threadIdx.x; i0 < kAll || !staged; i0 += N * step) {
    uint4 v[N], w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + k * step, u = i % U, r = i / U % R, h = i / (U * R);
      if (i < kAll && r < rows && h < heads) {
        int c0, c1;
        rope_chunks(t, u, c0, c1);
        const uint16_t* from = x + r * xr + h * xh;
        v[k] = *reinterpret_cast<const uint4*>(from + c0);
        w[k] = *reinterpret_cast<const uint4*>(from + c1);
      }
    }
    if (!staged) {
      rope_stage(t, turns, rows, inverse, status, pos);
      __syncthreads();
      staged = true;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + k * step, u = i % U, r = i / U % R, h = i / (U * R);
      if (i < kAll && r < rows && h < heads) {
        int c0, c1;
        rope_chunks(t, u, c0, c1);
        if (u < (t.pairs >> 3)) {
          float f[8], g[8];
          rope_apply(t, turns + r * kRopeRow, u, v[k], w[k], f, g);
          v[k] = bf16_of(f);
          w[k] = bf16_of(g);
        }
        uint16_t* to = y + r * yr + h * yh;
        *reinterpret_cast<uint4*>(to + c0) = v[k];
        *reinterpret_cast<uint4*>(to + c1) = w[k];
      }
    }
  }
}

}  // namespace
}  // namespace kvq
