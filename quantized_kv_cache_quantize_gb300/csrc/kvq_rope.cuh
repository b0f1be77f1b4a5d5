// Device helpers of the rotary positions: rows' positions, cosines and sines
// from the table, the rotation itself.
#pragma once

#include "kvq_checks.cuh"
#include "kvq_pages.cuh"

namespace kvq {
namespace {

// the axis of pair p.  (By selection: an address among the kernel's parameters that
// each lane computes for itself is a slow load.)
__device__ __forceinline__ int rope_axis(const RopeTab& t, int p) {
  const uint32_t w = p < 32 ? (p < 16 ? t.axis[0] : t.axis[1]) : (p < 48 ? t.axis[2] : t.axis[3]);
  return (int)((w >> (2 * (p & 15))) & 3u);
}
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
__device__ __forceinline__ void rope_stage_one(const RopeTab& t, float4* row, int* status, int* site, Pos pos,
                                               bool inverse = false) {
  const int e = threadIdx.x & 31, p = 2 * e;
  if (p >= t.pairs) return;
  const int axis0 = rope_axis(t, p), axis1 = rope_axis(t, p + 1);
  const float2* from = t.cs + (long long)rope_position(t, pos(axis0), status) * t.pairs + p;
  if (!KVQ_IN_BOUNDS(from - t.cs, (long long)t.n * t.pairs - 1, status, site)) return;
  float4 v;   // cos, sin, cos, sin
  if (axis0 == axis1) {
    v = __ldg(reinterpret_cast<const float4*>(from));
  } else {
    const float2* other = t.cs + (long long)rope_position(t, pos(axis1), status) * t.pairs + p + 1;
    if (!KVQ_IN_BOUNDS(other - t.cs, (long long)t.n * t.pairs, status, site)) return;
    const float2 x = __ldg(from), y = __ldg(other);
    v = make_float4(x.x, x.y, y.x, y.y);
  }
  row[rope_slot(e >> 2, e & 3)] = inverse ? make_float4(v.x, v.z, -v.y, -v.w) : make_float4(v.x, v.z, v.y, v.w);
}
// Those of `rows` rows by a block, a warp a row.  pos(row, axis): a row's position.
template <typename Pos>
__device__ __forceinline__ void rope_stage(const RopeTab& t, float4* turns, int rows, bool inverse, int* status, int* site,
                                           Pos pos) {
  for (int r = threadIdx.x >> 5; r < rows; r += blockDim.x >> 5)
    rope_stage_one(t, turns + r * kRopeRow, status, site, [&](int axis) { return pos(r, axis); }, inverse);
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

// Two pairs: a, b their first and second channels.  Each product and sum is
// rounded by itself: the bits are those of the formula evaluated step by step in
// fp32, whatever else a kernel does around it.  The products are fused with a -0
// that the compiler does not know (`none` of the call's table): it would make a
// plain product on pairs and the sum behind it one operation, rounded once.
__device__ __forceinline__ void turn_pairs(uint64_t a, uint64_t b, const float4& cs, uint64_t none, uint64_t& y0, uint64_t& y1) {
  const uint64_t c = ptx::f2_pack(cs.x, cs.y), s = ptx::f2_pack(cs.z, cs.w);
  y0 = ptx::f2_sub(ptx::f2_fma(a, c, none), ptx::f2_fma(b, s, none));
  y1 = ptx::f2_add(ptx::f2_fma(b, c, none), ptx::f2_fma(a, s, none));
}

// 16 channels of a row, unit u of d / 16: where u < pairs / 8, the channels of
// pairs [8 u, 8 u + 8) in two 16-byte chunks, rotated; behind them 16 channels
// that stay.  `c0`, `c1`: the chunks, in elements.
__device__ __forceinline__ void rope_chunks(const RopeTab& t, int u, int& c0, int& c1) {
  const bool halves = u < (t.pairs >> 3) && !t.interleaved;
  c0 = halves ? 8 * u : 16 * u;
  c1 = halves ? c0 + t.pairs : c0 + 8;
}
// The unit's chunks a, b as fp32 f, g, rotated by its entries of the row's turns.
// Interleaved pairs are the words of the chunks, the others a word of each.
template <bool INTER>
__device__ __forceinline__ void rope_apply(const RopeTab& t, const float4 (&cs)[4], const uint4& a, const uint4& b,
                                           float (&f)[8], float (&g)[8]) {
  const uint64_t none = ptx::f2_pack(t.none, t.none);
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t y0, y1;
    if (INTER) {
      const uint32_t w0 = j < 2 ? wa[2 * j] : wb[2 * j - 4], w1 = j < 2 ? wa[2 * j + 1] : wb[2 * j - 3];
      turn_pairs(ptx::f2_pack(lo(w0), lo(w1)), ptx::f2_pack(hi(w0), hi(w1)), cs[j], none, y0, y1);
      if (j < 2) {
        ptx::f2_unpack(y0, f[4 * j], f[4 * j + 2]);
        ptx::f2_unpack(y1, f[4 * j + 1], f[4 * j + 3]);
      } else {
        ptx::f2_unpack(y0, g[4 * j - 8], g[4 * j - 6]);
        ptx::f2_unpack(y1, g[4 * j - 7], g[4 * j - 5]);
      }
    } else {
      turn_pairs(ptx::f2_pack(lo(wa[j]), hi(wa[j])), ptx::f2_pack(lo(wb[j]), hi(wb[j])), cs[j], none, y0, y1);
      ptx::f2_unpack(y0, f[2 * j], f[2 * j + 1]);
      ptx::f2_unpack(y1, g[2 * j], g[2 * j + 1]);
    }
  }
}
__device__ __forceinline__ void rope_entries(const float4* row, int u, float4 (&cs)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) cs[j] = row[rope_slot(u, j)];
}

// R rows of up to kRopeHeads heads of one tensor by a block, whose threads are a
// multiple of R * D / 16: a thread has one unit of one row, of N heads at a time.
// The values are asked for first, then the rows' turns go through shared memory
// (R * kRopeRow), read once for all heads.  x, y: row 0, head 0.
template <int D, int R, int N, bool INTER, typename Pos>
__device__ __forceinline__ void rope_tile(const RopeTab& t, bool inverse, float4* turns, int rows, int heads,
                                          const uint16_t* x, long long xr, long long xh, uint16_t* y, long long yr,
                                          long long yh, int* status, int* site, Pos pos) {
  constexpr int U = D / 16;
  const int u = threadIdx.x % U, r = threadIdx.x / U % R, step = blockDim.x / (R * U);
  const bool live = r < rows, turned = u < (t.pairs >> 3);
  int c0, c1;
  rope_chunks(t, u, c0, c1);
  x += r * xr;
  y += r * yr;
  float4 cs[4];
  bool staged = false;
  for (int h0 = threadIdx.x / (R * U); h0 < heads || !staged; h0 += N * step) {
    uint4 v[N], w[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int h = h0 + k * step;
      if (live && h < heads) {
        const uint16_t* from = x + h * xh;
        v[k] = *reinterpret_cast<const uint4*>(from + c0);
        w[k] = *reinterpret_cast<const uint4*>(from + c1);
      }
    }
    if (!staged) {
      rope_stage(t, turns, rows, inverse, status, site, pos);
      __syncthreads();
      staged = true;
      if (live && turned) rope_entries(turns + r * kRopeRow, u, cs);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int h = h0 + k * step;
      if (live && h < heads) {
        if (turned) {
          float f[8], g[8];
          rope_apply<INTER>(t, cs, v[k], w[k], f, g);
          v[k] = bf16_of(f);
          w[k] = bf16_of(g);
        }
        uint16_t* to = y + h * yh;
        *reinterpret_cast<uint4*>(to + c0) = v[k];
        *reinterpret_cast<uint4*>(to + c1) = w[k];
      }
    }
  }
}

}  // namespace
}  // namespace kvq
