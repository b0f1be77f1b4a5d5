// Device helpers of the rotary positions: rows' positions, cosines and sines
// from the table, the rotation itself.
#pragma once

#include "kvq_pages.cuh"

namespace kvq {
namespace {

// The positions of a row, each held inside the table (a position outside it is
// recorded).
struct RopeAt {
  int p[kRopeMaxAxes];
};
__device__ __forceinline__ int rope_position(const RopeTab& t, int p, int* status) {
  if ((unsigned)p >= (unsigned)t.n) {
    atomicCAS(status, 0, (int)KVQ_ERR_POSITION);
    p = min(max(p, 0), t.n - 1);
  }
  return p;
}
__device__ __forceinline__ RopeAt rope_at(const RopeTab& t, const int32_t* pos, long long axis_stride, int* status) {
  RopeAt at;
#pragma unroll
  for (int k = 0; k < kRopeMaxAxes; ++k) at.p[k] = k < t.axes ? rope_position(t, __ldg(pos + k * axis_stride), status) : 0;
  return at;
}
__device__ __forceinline__ RopeAt rope_at(const RopeTab& t, int pos, int* status) {
  RopeAt at;
  at.p[0] = rope_position(t, pos, status);
#pragma unroll
  for (int k = 1; k < kRopeMaxAxes; ++k) at.p[k] = at.p[0];
  return at;
}

// (cos, sin) of pairs [p0, p0 + N)
template <int N>
__device__ __forceinline__ void rope_turn(const RopeTab& t, const RopeAt& at, int p0, bool inverse, float2 (&cs)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int axis = t.axis[p0 + k];
    const int pos = axis == 0 ? at.p[0] : axis == 1 ? at.p[1] : axis == 2 ? at.p[2] : at.p[3];
    cs[k] = __ldg(t.cs + (long long)pos * t.pairs + p0 + k);
    if (inverse) cs[k].y = -cs[k].y;
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
__device__ __forceinline__ void rope_apply(const RopeTab& t, const float2 (&cs)[8], uint4& a, uint4& b) {
  float x[8], y[8], u[8], v[8];
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
  a = bf16_of(u);
  b = bf16_of(v);
}

}  // namespace
}  // namespace kvq
