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

// Turns of rows in shared memory, kRopeRow numbers (cos, sin) a row: pair p stands
// where the threads of a row's units (of 8 pairs) read 16 bytes each that are
// neighbours, so that they meet different banks.
constexpr int kRopeRow = kRopeMaxPairs;
__device__ __forceinline__ int rope_slot(int p) { return ((p & 7) >> 1) * 16 + (p >> 3) * 2 + (p & 1); }
// Fills those of `rows` rows, a pair a thread: neighbouring pairs of an axis are
// neighbours in the table too.  pos(row, axis): a row's position.
template <typename Pos>
__device__ __forceinline__ void rope_stage(const RopeTab& t, float2* turns, int rows, bool inverse, int* status, Pos pos) {
  for (int i = threadIdx.x; i < rows * kRopeRow; i += blockDim.x) {
    const int r = i / kRopeRow, p = i % kRopeRow;
    if (p >= t.pairs) continue;
    const int at = rope_position(t, pos(r, (int)t.axis[p]), status);
    float2 cs = __ldg(t.cs + (long long)at * t.pairs + p);
    if (inverse) cs.y = -cs.y;
    turns[r * kRopeRow + rope_slot(p)] = cs;
  }
}
// the turns of unit u of a row
__device__ __forceinline__ void rope_turns(const float2* row, int u, float2 (&cs)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(row + j * 16 + u * 2);
    cs[2 * j] = make_float2(v.x, v.y);
    cs[2 * j + 1] = make_float2(v.z, v.w);
  }
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

// Each product and sum rounded by itself: the bits are those of the formula
// evaluated step by step in fp32, whatever else a kernel does around it.
__device__ __forceinline__ float turn_first(float x0, float x1, float2 cs) {
  return __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y));
}
__device__ __forceinline__ float turn_second(float x0, float x1, float2 cs) {
  return __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, cs.y));
}

// 16 channels of a row, unit u of d / 16: where u < pairs / 8, the channels of
// pairs [8 u, 8 u + 8) in two 16-byte chunks, rotated; behind them 16 channels
// that stay.  `c0`, `c1`: the chunks, in elements.
__device__ __forceinline__ void rope_chunks(const RopeTab& t, int u, int& c0, int& c1) {
  const bool halves = u < (t.pairs >> 3) && !t.interleaved;
  c0 = halves ? 8 * u : 16 * u;
  c1 = halves ? c0 + t.pairs : c0 + 8;
}
__device__ __forceinline__ void rope_apply(const RopeTab& t, const float2 (&cs)[8], const uint4& a, const uint4& b,
                                           float (&u)[8], float (&v)[8]) {
  float x[8], y[8];
  floats_of(a, x);
  floats_of(b, y);
  if (t.interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[2 * k] = turn_first(x[2 * k], x[2 * k + 1], cs[k]);
      u[2 * k + 1] = turn_second(x[2 * k], x[2 * k + 1], cs[k]);
      v[2 * k] = turn_first(y[2 * k], y[2 * k + 1], cs[4 + k]);
      v[2 * k + 1] = turn_second(y[2 * k], y[2 * k + 1], cs[4 + k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      u[k] = turn_first(x[k], y[k], cs[k]);
      v[k] = turn_second(x[k], y[k], cs[k]);
    }
  }
}

// R rows of up to kRopeHeads heads of one tensor by a block: the values are asked
// for first, then the rows' turns go through shared memory (R * kRopeRow), read
// once for all heads.  x, y: row 0, head 0.
constexpr int kRopeHeads = 8;
template <int D, int R, typename Pos>
__device__ __forceinline__ void rope_tile(const RopeTab& t, bool inverse, float2* turns, int rows, int heads,
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
          float2 cs[8];
          float f[8], g[8];
          rope_turns(turns + r * kRopeRow, u, cs);
          rope_apply(t, cs, v[k], w[k], f, g);
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
