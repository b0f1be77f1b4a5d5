// Attention over the paged cache for few query rows per sequence (the rows of a
// cache head: its group of query heads times the sequence's query tokens), the
// form of a decoding step, up to 16 rows.
//
// Per (sequence, cache head): s_j = c q . k_j, one pass over the keys with the
// running maximum and sum of the softmax.  The keys are read once for all
// rows of the head, so the pass is bound by the cache's bytes (2 d per key and
// head against 4 d rows flops: at 16 rows 32 flops per byte, far below the
// tensor cores' 280).  What costs next is the work per byte: codes to FP16,
// 16-bit products, exponentials.
//
// Work split.  The keys of all (sequence, head) items, in units of 32, are one
// long line; every warp of the grid takes an equal run of it, whatever the
// lengths of the batch.  A warp works alone: its own ring of TMA stages in
// shared memory (each lane-0 copies a unit's K and V rows, swizzled, from the
// page), its own running softmax, no barrier with other warps.  An item that
// one warp covers is written by it; the parts of the others go to the
// workspace and a second, small kernel joins them in order (no atomics, the
// same bits every time).
//
// Products.  mma.sync m16n8k16 with the keys as the 16 rows and up to 8 query
// rows as the columns: S^T = K Q^T, then O^T = V^T P^T.  Both read the codes
// straight from shared memory into fragment layout, because a contraction may
// take its terms in any order: a lane's 16 bytes of a key row are the K
// fragment of four k-steps (the query fragment permuted alike), and two rows'
// bytes interleaved by one byte permute are the V^T fragment.  A tcgen05
// product would need the codes converted and stored to shared memory again
// for a tile that has 16 of 128 rows filled.  E4M3 products (m16n8k32, the
// query in high and low parts) would spare the conversion of K, but measured
// slower: 249 against 188 us for 16 rows, 32 sequences of 16384 keys, 8 heads.
//
// Numbers.  E4M3 codes are exact in FP16.  A query row is scaled by a power of
// two to a largest magnitude in [2^14, 2^15): exact in FP16 down to 2^-31 of
// that maximum, off by 2^-39 of it at most below.  The page scales are powers of two applied outside the
// products: K's to the fp32 scores, V's (2^ev) to the weight before it is
// rounded to FP16.  Two running bases a row, over the keys that it attends to:
// the largest score m for the sum of weights, which knows no V scale, and the
// largest score plus ev, held as m + eo, for the output.  The largest product
// of a weight and its scale stands at 2^15 in FP16, so products down to 2^-39
// of it remain, whatever the scales of pages that carry less, or that other
// rows see.  A second exponential a score keeps the sum exact at any distance
// of the two bases; the special-function unit is idle enough, and the maxima
// of the eight row groups meet only where a base rises (64 sequences of up to
// 8192 keys: 83 us either way).
//
// Shaped scores (MODE, kvq_scores.cuh) cost nothing that HBM does not hide: the
// same 64 sequences with a bias 80 to 82 us; 4 of 100001 keys, 40 heads over 8, with
// a cap 142 to 147, without 141.  An item's keys run from the first to the last that
// a row of it attends to; a key between them that none does (documents) keeps its
// value out of the product by a vote of the lanes that hold its scores.
#pragma once

#include <math_constants.h>

#include "kvq_checks.cuh"
#include "kvq_pages.cuh"
#include "kvq_scores.cuh"

namespace kvq {
namespace {

constexpr int kUnit = 32;          // keys per unit
constexpr int kMinUnits = 2;       // per warp, when the work is small
// What an item's start costs the warp that comes to it from another one, in
// units: its table entries, scales, query rows and first copies one after
// another (64 sequences of up to 8192 keys, 8 heads: none 96.7, one 87.9, two
// 85.1, three 85.1 us).
constexpr int kStartUnits = 2;
constexpr int kMaxCluster = 16;
constexpr float kNoOutput = -1000.f;   // where a row's output has no base yet

// W warps per CTA, one CTA per SM
template <int D, int W>
struct DecCfg {
  static constexpr int kWarps = W;
  static constexpr int kHalf = kUnit * D;                 // K (or V) rows of a unit
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 196608 / (kWarps * kStage);   // per warp; 192 KB in all
  static constexpr int kBar = kWarps * kStages * kStage;
  static constexpr int kBytes = kBar + kWarps * kStages * 8;
  static constexpr int kAlloc = kBytes + 1024;
};

struct DecodeArgs {
  PagedAttnArgs a;
  long long* pre;      // [batch + 1] first unit of each sequence (written by CTA 0)
  float* part_o;       // [2 warps][rows_cap][D]
  float* part_ml;      // [2 warps][rows_cap][2]
  int rows_cap;        // rows of an item at most: max_q * group, up to 8 NT
  int warps;           // of the grid
  int cluster;         // CTAs per item (decode_item_kernel)
};

// What sequence b has to do: its rows, keys [lo, len) that any row attends to
// (lo rounded down to a unit), units of a cache head.
struct SeqWork {
  int r0, n, len, lo, units;
  int seen;   // first key some row attends to; lo is this rounded down
  int end;    // no row attends to a key from here on
};
template <int MODE>
__device__ __forceinline__ SeqWork seq_work(const PagedAttnArgs& a, int b) {
  SeqWork w;
  seq_rows(a.s, b, w.r0, w.n, a.status);
  if (w.n > a.max_q) {
    page_error(a.status);
    w.n = a.max_q;
  }
  w.len = seq_len(a.s, b, a.p.shift, a.status);
  const int t0 = w.len - w.n;
  w.seen = a.window > 0 ? max(0, t0 - a.window + 1) : 0;
  w.end = w.len;
  if (MODE != kPlain) {
    int lo = w.len, hi = 0;
    for (int i = 0; i < w.n; ++i) {
      const RowView v = row_view(a, b, w.r0 + i, t0 + i, w.len);
      if (v.lo < v.hi) {
        lo = min(lo, v.lo);
        hi = max(hi, v.hi);
      }
    }
    w.seen = min(lo, hi);
    w.end = hi;
  }
  w.lo = w.seen & ~(kUnit - 1);
  // a sequence with rows has one unit at least: it writes their empty result
  w.units = w.n > 0 ? max(1, (w.end - w.lo + kUnit - 1) / kUnit) : 0;
  return w;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t lo_f16(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)w); }
__device__ __forceinline__ uint32_t hi_f16(uint32_t w) { return f16x2_of_e4m3x2((uint16_t)(w >> 16)); }
__device__ __forceinline__ void lds128(uint32_t (&w)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void lds64(uint32_t (&w)[2], uint32_t addr) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}

// key row (of 8) that fragment row j holds: even rows 0 2 4 6, odd rows those
// xor 5, so that the rows a quarter-warp reads together meet different banks
// of the swizzled tile, both as K rows (pairs j, j + 1) and as V rows (all
// even, then all odd j)
__device__ __forceinline__ int key_row(int j) { return (j & 6) ^ ((j & 1) * 5); }

// A warp's ring of stages and where it stands.
struct Ring {
  uint32_t data, bars;
  int stage;
  uint32_t phase;
};

// Raw scores of 16 keys capped, in units of the cap.
template <int NT>
__device__ __forceinline__ void cap_scores(float (&s)[NT][4], const float (&cq)[NT][2], float fk) {
  float top = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      s[nt][c] *= cq[nt][c & 1] * fk;
      top = fmaxf(top, fabsf(s[nt][c]));
    }
  const bool far = __any_sync(0xffffffffu, top > 1.f);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      float x, y;
      ptx::f2_unpack(tanh_small(ptx::f2_pack(s[nt][c], s[nt][c + 1])), x, y);
      s[nt][c] = far ? tanh_any(s[nt][c], x) : x;
      s[nt][c + 1] = far ? tanh_any(s[nt][c + 1], y) : y;
    }
}

// One segment: units [i0, i0 + seg) of (b, h), by one warp.  o, m, l: for the
// rows nt * 8 + 2 t + c (c = 0, 1) the channels CH g .. of sum p v (channel
// 2 k + i in o[nt][k][c + 2 i]), the base in units of log 2 and sum p.  False
// when a wait ran out.
template <int D, int NT, int W, int MODE>
__device__ __forceinline__ bool decode_segment(const PagedAttnArgs& a, const CUtensorMap& map_k,
                                               const CUtensorMap& map_v, Ring& rg, int b, int h,
                                               const SeqWork& w, int i0, int seg,
                                               float (&o)[NT][D / 16][4], float (&m)[NT][2],
                                               float (&l)[NT][2]) {
  using C = DecCfg<D, W>;
  constexpr int KC = D / 64;       // 16-byte chunks of a key row per lane
  constexpr int MT = D / 16;       // channel tiles of the output
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, heads = a.p.heads;
  const float scale_log2 = raw_factor<MODE>(a);   // (of the cap, in a capped mode)
  const uint32_t ring = rg.data, bars = rg.bars;
  int& stage = rg.stage;
  uint32_t& phase = rg.phase;
  const int rows = w.n * a.group;
  const int key_first = w.lo + i0 * kUnit;
  const int key_end = min(w.end, w.lo + (i0 + seg) * kUnit);
  const int t0 = w.len - w.n;
  // ---- the query rows' loads, first: their latency runs beside the table's ----
  uint2 raw[NT][KC * 4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
#pragma unroll
    for (int k = 0; k < KC * 4; ++k) raw[nt][k] = make_uint2(0u, 0u);
    if (r < rows) {
      const int i = r / a.group, hq = h * a.group + r % a.group;
      const uint16_t* qp = a.q + (long long)(w.r0 + i) * a.q_row_stride + (long long)hq * a.q_head_stride;
#pragma unroll
      for (int k = 0; k < KC; ++k) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(qp + 16 * (t + 4 * k)) + v);
          raw[nt][4 * k + 2 * v] = make_uint2(x.x, x.y);
          raw[nt][4 * k + 2 * v + 1] = make_uint2(x.z, x.w);
        }
      }
    }
  }
  // pages, 32 at a time, one per lane: id (-1: none), exponents of K and V
  const int shift = a.p.shift;
  const int page_end = (max(key_end, key_first) + a.p.page - 1) >> shift;
  int pbase = key_first >> shift;
  auto page_info = [&](int base, int& id, int& ek, int& ev) {
    id = -1;
    ek = ev = 0;
    // (a page wholly before every row's window may be gone already)
    if (base + lane < page_end && ((long long)(base + lane + 1) << shift) > w.seen) {
      id = seq_page(a.s, b, base + lane, a.p.n_pages, a.status);
      if (id >= 0) {
        const long long blk = (long long)id * heads + h;
        ek = scale_exp(__ldg(a.p.scale[0] + blk));
        ev = scale_exp(__ldg(a.p.scale[1] + blk));
      }
    }
  };
  int id0, ek0, ev0, id1, ek1, ev1;
  page_info(pbase, id0, ek0, ev0);
  page_info(pbase + 32, id1, ek1, ev1);
  auto pick = [&](int v0, int v1, int pg) {
    const int r = pg - pbase;
    const int x = __shfl_sync(0xffffffffu, v0, r & 31), y = __shfl_sync(0xffffffffu, v1, r & 31);
    return r < 32 ? x : y;
  };
  // copy unit i of the segment into stage st (all lanes; lane 0 issues)
  auto fetch = [&](int i, int st) {
    const int key0 = key_first + i * kUnit;
    const uint32_t dst = ring + (uint32_t)(st * C::kStage), bar = bars + 8u * st;
    const int pg = key0 >> shift;
    const int ida = pick(id0, id1, pg);
    const bool two = shift == 4;
    const int idb = two ? pick(id0, id1, pg + 1) : -1;
    if (lane == 0) {
      const int box = two ? 16 : 32;
      const bool la = ida >= 0 && key0 < key_end, lb = idb >= 0 && key0 + 16 < key_end;
      const uint32_t bytes = (uint32_t)(2 * box * D) * ((la ? 1u : 0u) + (lb ? 1u : 0u));
      if (bytes == 0) {
        ptx::mbar_arrive(bar);
      } else {
        ptx::mbar_expect_tx(bar, bytes);
        const int in = key0 & (a.p.page - 1);
        if (la) {
          ptx::tma_load_3d(dst, &map_k, 0, in, ida * heads + h, bar);
          ptx::tma_load_3d(dst + C::kHalf, &map_v, 0, in, ida * heads + h, bar);
        }
        if (lb) {
          ptx::tma_load_3d(dst + 16 * D, &map_k, 0, 0, idb * heads + h, bar);
          ptx::tma_load_3d(dst + C::kHalf + 16 * D, &map_v, 0, 0, idb * heads + h, bar);
        }
      }
    }
  };
  const int ahead = min(seg, C::kStages);
  for (int i = 0; i < ahead; ++i) fetch(i, (stage + i) % C::kStages);

  // ---- query rows as B fragments, scaled to FP16 ----
  uint32_t qf[NT][KC * 4][2];
  float cq[NT][2];
  int lo_r[NT][2], hi_r[NT][2];   // keys each column's row attends to
  int ref[NT][2];                 // where its distances are counted from
  RowShape shape[NT][2];
  int every_lo = 0, every_hi = 0x7fffffff;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    uint32_t mx = 0;   // largest magnitude, as its bits
#pragma unroll
    for (int k = 0; k < KC * 4; ++k) {
      mx = max(mx, max(max((raw[nt][k].x & 0x7fffu), (raw[nt][k].x >> 16) & 0x7fffu),
                       max((raw[nt][k].y & 0x7fffu), (raw[nt][k].y >> 16) & 0x7fffu)));
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the maximum's exponent becomes 14 (a subnormal maximum's at most)
    const int e = max((int)(mx >> 7), 1) - 127 - 14;
    // x * 2^-e in two steps, each factor a normal number
    // (an infinity or a NaN makes the whole row NaN)
    const float f0 = mx < 0x7f80u ? pow2f(-(e / 2)) : CUDART_NAN_F, f1 = pow2f(-(e - e / 2));
#pragma unroll
    for (int k = 0; k < KC * 4; ++k) {
      qf[nt][k][0] = ptx::f16x2_rn(__uint_as_float(raw[nt][k].x << 16) * f0 * f1, __uint_as_float(raw[nt][k].x & 0xffff0000u) * f0 * f1);
      qf[nt][k][1] = ptx::f16x2_rn(__uint_as_float(raw[nt][k].y << 16) * f0 * f1, __uint_as_float(raw[nt][k].y & 0xffff0000u) * f0 * f1);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      // column 2t + c is the row whose lanes have g = 2t + c
      const int ec = __shfl_sync(0xffffffffu, e, (2 * t + c) * 4);
      cq[nt][c] = scale_log2 * pow2f(ec / 2) * pow2f(ec - ec / 2);
      const int rc = nt * 8 + 2 * t + c;
      const int tq = t0 + rc / a.group;
      if (MODE == kPlain) {
        hi_r[nt][c] = rc < rows ? (a.causal ? min(w.len, tq + 1) : w.len) : 0;
        lo_r[nt][c] = a.window > 0 ? max(0, tq - a.window + 1) : 0;
      } else {
        hi_r[nt][c] = lo_r[nt][c] = ref[nt][c] = 0;
        shape[nt][c] = RowShape{};
        if (rc < rows) {
          const RowView v = row_view(a, b, w.r0 + rc / a.group, tq, w.len);
          hi_r[nt][c] = v.hi;
          lo_r[nt][c] = v.lo;
          ref[nt][c] = v.ref;
          shape[nt][c] = row_shape<MODE>(a, h * a.group + rc % a.group);
          every_lo = max(every_lo, v.lo);
          every_hi = min(every_hi, v.hi);
        }
      }
    }
  }
  if (MODE != kPlain) {
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      every_lo = max(every_lo, __shfl_xor_sync(0xffffffffu, every_lo, x));
      every_hi = min(every_hi, __shfl_xor_sync(0xffffffffu, every_hi, x));
    }
  }
  // keys every row attends to
  const int all_lo = MODE != kPlain ? every_lo : a.window > 0 ? max(0, w.len - a.window) : 0;
  const int all_hi = MODE != kPlain ? every_hi : a.causal ? min(w.len, t0 + 1) : w.len;

#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
    m[nt][0] = m[nt][1] = -CUDART_INF_F;
    l[nt][0] = l[nt][1] = 0.f;
  }
  float eo[NT][2];    // O is held against m + eo (see the head of this file)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) eo[nt][0] = eo[nt][1] = kNoOutput;
  bool ok = true;

  for (int i = 0; i < seg; ++i) {
    const int key0 = key_first + i * kUnit;
    ok = page_wait(bars + 8u * stage, phase, a.wait_limit_ns, nullptr, a.status);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    if ((key0 >> shift) - pbase >= 32) {
      pbase += 32;
      id0 = id1, ek0 = ek1, ev0 = ev1;
      page_info(pbase + 32, id1, ek1, ev1);
    }
    const uint32_t kb = ring + (uint32_t)(stage * C::kStage), vb = kb + C::kHalf;
    // one key per 16-row tile decides its page: tiles never straddle pages
    int idt[2], ekt[2], evt[2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const int pg = (key0 + 16 * mt) >> shift;
      idt[mt] = pick(id0, id1, pg);
      ekt[mt] = pick(ek0, ek1, pg);
      evt[mt] = pick(ev0, ev1, pg);
    }
    const bool whole = key0 >= all_lo && key0 + kUnit <= all_hi && idt[0] >= 0 && idt[1] >= 0;

    // ---- S^T = K Q^T ----
    float s[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[mt][nt][c] = 0.f;
      const int ra = 16 * mt + key_row(g);
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        uint32_t x[4], y[4];
        uint32_t off;
        if (D == 128) off = (uint32_t)(ra * 128 + (((t + 4 * k) ^ (ra & 7)) << 4));
        else off = (uint32_t)(ra * 64 + ((t ^ ((ra >> 1) & 3)) << 4));
        lds128(x, kb + off);
        lds128(y, kb + off + 8 * D);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint32_t a0 = lo_f16(x[v]), a1 = lo_f16(y[v]), a2 = hi_f16(x[v]), a3 = hi_f16(y[v]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(s[mt][nt], a0, a1, a2, a3, qf[nt][4 * k + v][0], qf[nt][4 * k + v][1]);
        }
      }
    }
    // ---- softmax ----
    // the lane's largest score of a column among each tile's keys
    float xm[2][NT][2];
    uint32_t some[2][2];   // lanes whose key (of tile, of its half) a row of theirs attends to
    const float ev[2] = {(float)evt[0], (float)evt[1]};
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      const float fk = pow2f(ekt[mt]);
      const int ka = key0 + 16 * mt + key_row(g);
      bool mine[2] = {false, false};
      if (MODE == kCapped) cap_scores<NT>(s[mt], cq, fk);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        xm[mt][nt][0] = xm[mt][nt][1] = -CUDART_INF_F;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v = MODE == kCapped ? s[mt][nt][c] * shape[0][0].cap2 : s[mt][nt][c] * (cq[nt][c & 1] * fk);
          if (MODE != kPlain && shape[0][0].biased)
            v = fmaf(-shape[nt][c & 1].slope2, (float)abs(ref[nt][c & 1] - (ka + 8 * (c >> 1))), v);
          if (!whole) {
            const int key = ka + 8 * (c >> 1);
            const bool see = key >= lo_r[nt][c & 1] && key < hi_r[nt][c & 1] && idt[mt] >= 0;
            v = see ? v : -CUDART_INF_F;
            mine[c >> 1] |= see;
          }
          s[mt][nt][c] = v;
          xm[mt][nt][c & 1] = fmaxf(xm[mt][nt][c & 1], v);
        }
      }
      if (MODE != kPlain && !whole) {
        some[mt][0] = __ballot_sync(0xffffffffu, mine[0]);
        some[mt][1] = __ballot_sync(0xffffffffu, mine[1]);
      }
    }
    // (a score plus ev is looked at through its distance from m, which is
    // exact near m however large the scores)
    bool grows = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
          grows |= xm[mt][nt][c] > m[nt][c] || (xm[mt][nt][c] - m[nt][c]) + ev[mt] > eo[nt][c];
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(xm[0][nt][c], xm[1][nt][c]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float mn = fmaxf(m[nt][c], top);
          const bool any = mn > -CUDART_INF_F;     // the row attends to something so far
          const float mb = any ? mn : 0.f, down = any ? m[nt][c] - mn : 0.f;
          float en = fmaxf((xm[0][nt][c] - mb) + ev[0], (xm[1][nt][c] - mb) + ev[1]);
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) en = fmaxf(en, __shfl_xor_sync(0xffffffffu, en, x));
          en = fmaxf(en, eo[nt][c] + down);
          l[nt][c] *= ptx::ex2_approx(down);
          f[c] = ptx::ex2_approx(down + (eo[nt][c] - en));
          m[nt][c] = mn;
          eo[nt][c] = en;
        }
#pragma unroll
        for (int k = 0; k < MT; ++k)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[nt][k][c] *= f[c & 1];
      }
    }
    // ---- weights: P^T as B fragments ----
    uint32_t pf[2][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] > -CUDART_INF_F ? m[nt][0] : 0.f, m1 = m[nt][1] > -CUDART_INF_F ? m[nt][1] : 0.f;
      const uint64_t mb = ptx::f2_pack(m0, m1);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint64_t up = ptx::f2_pack((ev[mt] - eo[nt][0]) + 15.f, (ev[mt] - eo[nt][1]) + 15.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t x = ptx::f2_sub(ptx::f2_pack(s[mt][nt][2 * i], s[mt][nt][2 * i + 1]), mb);
          float x0, x1, w0, w1;
          ptx::f2_unpack(x, x0, x1);
          l[nt][0] += ptx::ex2_approx(x0);
          l[nt][1] += ptx::ex2_approx(x1);
          ptx::f2_unpack(ptx::f2_add(x, up), w0, w1);
          pf[mt][nt][i] = transpose8x8(ptx::f16x2_rn(ptx::ex2_approx(w0), ptx::ex2_approx(w1)));
        }
      }
    }
    // ---- O^T += V^T P^T ----
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      // rows of fragment columns 2t, 2t + 1, 2t + 8, 2t + 9
      const int rv[2] = {key_row(2 * t), key_row(2 * t + 1)};
      uint32_t x[4][D / 32];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 16 * mt + rv[j & 1] + 8 * (j >> 1);
        if constexpr (D == 128) lds128(x[j], vb + (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4)));
        else lds64(x[j], vb + (uint32_t)(r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8));
        if (!whole) {
          // what no row of the sequence may see must not reach the product
          // (a zero weight times a NaN)
          const int key = key0 + r;
          bool use = key >= w.seen && key < w.len && idt[mt] >= 0;
          // (between ranges there may be keys that no row attends to: key_row(g)
          // is the key of lanes 4 g .. 4 g + 3, which hold all rows)
          if (MODE != kPlain) use = use && ((some[mt][j >> 1] >> (4 * (2 * t + (j & 1)))) & 15u) != 0u;
#pragma unroll
          for (int v = 0; v < D / 32; ++v) x[j][v] = use ? x[j][v] : 0u;
        }
      }
#pragma unroll
      for (int v = 0; v < D / 32; ++v) {
        const uint32_t ab0 = __byte_perm(x[0][v], x[1][v], 0x5140), ab1 = __byte_perm(x[0][v], x[1][v], 0x7362);
        const uint32_t cd0 = __byte_perm(x[2][v], x[3][v], 0x5140), cd1 = __byte_perm(x[2][v], x[3][v], 0x7362);
        const uint32_t f0 = lo_f16(ab0), f1 = hi_f16(ab0), f2 = lo_f16(cd0), f3 = hi_f16(cd0);
        const uint32_t e0 = lo_f16(ab1), e1 = hi_f16(ab1), e2 = lo_f16(cd1), e3 = hi_f16(cd1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma16816(o[nt][2 * v], f0, f1, f2, f3, pf[mt][nt][0], pf[mt][nt][1]);
          mma16816(o[nt][2 * v + 1], e0, e1, e2, e3, pf[mt][nt][0], pf[mt][nt][1]);
        }
      }
    }
    __syncwarp();
    if (i + ahead < seg) fetch(i + ahead, stage);
    if (++stage == C::kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (!ok) {
    // copies in flight still write this warp's stages: wait for them
    // (bounded) before it exits
    for (int i = 0; i < C::kStages; ++i) {
      page_drain(bars + 8u * stage, phase, a.wait_limit_ns);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
      if (i + 1 >= ahead) break;
    }
    return false;
  }
  // O in original units, the sums over the keys' lanes
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float fo = eo[nt][c] > kNoOutput ? ptx::ex2_approx(eo[nt][c] - 15.f) : 0.f;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        o[nt][k][c] *= fo;
        o[nt][k][c + 2] *= fo;
      }
    }
  return true;
}

// what a row's distance from its own keys adds to lse
template <int MODE>
__device__ __forceinline__ float row_bias(const PagedAttnArgs& a, const SeqWork& w, int b, int h, int r) {
  if (MODE == kPlain) return 0.f;
  const int i = r / a.group;
  return ref_bias(a, row_view(a, b, w.r0 + i, w.len - w.n + i, w.len), h * a.group + r % a.group);
}

// Row r of the head's rows, from the lane's share (lanes g hold channels
// CH g .., n = nt, c the row's place): BF16 out and lse.
template <int D, int NT, int MODE>
__device__ __forceinline__ void store_row(const PagedAttnArgs& a, const SeqWork& w, int b, int h, int r,
                                          const float (&o)[NT][D / 16][4], int nt, int c, float m, float l) {
  constexpr int CH = D / 8;
  const int g = (threadIdx.x & 31) >> 2;
  const long long row = (long long)(w.r0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
  if (!KVQ_IN_BOUNDS(row, (long long)a.s.rows * a.q_heads, a.status, a.bounds_site)) return;
  const float f = l == 0.f ? 0.f : 1.f / l;
  uint32_t v[CH / 2];
#pragma unroll
  for (int k = 0; k < CH / 2; ++k) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(o[nt][k][c] * f, o[nt][k][c + 2] * f);
    v[k] = *reinterpret_cast<const uint32_t*>(&z);
    if (MODE != kPlain && l == 0.f) v[k] = 0u;   // (zero weights times a NaN that other rows attend to)
  }
  uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + CH * g);
#pragma unroll
  for (int k = 0; k < CH / 8; ++k) dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  if (g == 0 && a.lse != nullptr)
    a.lse[row] = (l == 0.f ? -CUDART_INF_F : 0.6931471805599453f * (m + log2f(l))) + row_bias<MODE>(a, w, b, h, r);
}

template <int D, int NT, int W, int MODE>
__global__ void __launch_bounds__(W * 32, 1)
    decode_kernel(const __grid_constant__ DecodeArgs p, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using C = DecCfg<D, W>;
  constexpr int CH = D / 8;        // output channels per lane
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long scan_warp[C::kWarps];
  constexpr int kScan = C::kWarps * 32;
  __shared__ long long pre_s[kScan + 1];
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t ring = ptx::smem_u32(smem) + (uint32_t)(wid * C::kStages * C::kStage);
  const uint32_t bars = ptx::smem_u32(smem) + (uint32_t)(C::kBar + wid * C::kStages * 8);
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) ptx::mbar_init(bars + 8 * i, 1);
    ptx::fence_mbar_init();
  }
  ptx::grid_dependency_wait();
  ptx::launch_dependents();

  // ---- this warp's run of units ----
  const int heads = a.p.heads;
  // scan of one chunk of sequences: pre_s[i] = units before sequence c0 + i
  auto scan = [&](int c0, long long carry) -> long long {
    const int b = c0 + (int)threadIdx.x;
    long long v = 0;
    if (b < a.s.batch) {
      const SeqWork x = seq_work<MODE>(a, b);
      v = x.units > 0 ? (long long)(x.units + kStartUnits) * heads : 0;
    }
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) scan_warp[wid] = incl;
    __syncthreads();
    long long before = carry, all = carry;
#pragma unroll
    for (int w = 0; w < C::kWarps; ++w) {
      if (w < wid) before += scan_warp[w];
      all += scan_warp[w];
    }
    pre_s[threadIdx.x] = before + incl - v;
    if (threadIdx.x == 0) pre_s[kScan] = all;
    __syncthreads();
    return all;
  };
  long long total = 0;
  for (int c0 = 0; c0 < a.s.batch; c0 += kScan) {
    total = scan(c0, total);
    if (blockIdx.x == 0 && c0 + (int)threadIdx.x < a.s.batch) p.pre[c0 + threadIdx.x] = pre_s[threadIdx.x];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.pre[a.s.batch] = total;
  const long long per = max((total + p.warps - 1) / p.warps, (long long)kMinUnits);
  // neighbours in the line of units go to different SMs
  const int gw = wid * (int)gridDim.x + (int)blockIdx.x;
  const long long u0 = min((long long)gw * per, total), u1 = min(u0 + per, total);
  int b = 0;
  long long at = 0;   // first unit of sequence b
  {
    long long carry = 0;
    bool found = false;
    for (int c0 = 0; c0 < a.s.batch; c0 += kScan) {
      if (a.s.batch > kScan) carry = scan(c0, carry);
      const int n = min(kScan, a.s.batch - c0);
      // last sequence that starts at or before u0 (the empty ones among equal
      // starts are stepped over below)
      if (!found && u0 < pre_s[kScan]) {
        int l = 0, h = n - 1;
        while (l < h) {
          const int m = (l + h + 1) >> 1;
          if (pre_s[m] <= u0) l = m; else h = m - 1;
        }
        b = c0 + l;
        at = pre_s[l];
        found = true;
      }
    }
  }

  Ring rg{ring, bars, 0, 0u};
  SeqWork w{};
  if (u0 < u1) w = seq_work<MODE>(a, b);
  int h = 0, i0 = 0;
  if (u0 < u1) {
    h = (int)((u0 - at) / (w.units + kStartUnits));
    i0 = (int)((u0 - at) % (w.units + kStartUnits)) - kStartUnits;
  }
  for (long long u = u0; u < u1;) {
    if (i0 < 0) {   // the item's start
      u -= i0;
      i0 = 0;
      if (u >= u1) break;
    }
    const int seg = (int)min((long long)(w.units - i0), u1 - u);
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
    if (!decode_segment<D, NT, W, MODE>(a, map_k, map_v, rg, b, h, w, i0, seg, o, m, l)) break;
    // ---- its result: the item's, or a part of it ----
    const int rows = w.n * a.group;
    const bool complete = seg == w.units;
    const long long slot = 2LL * gw + (u == u0 ? 0 : 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        if (r >= rows) continue;
        if (complete) {
          store_row<D, NT, MODE>(a, w, b, h, r, o, nt, c, m[nt][c], l[nt][c]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (slot * p.rows_cap + r) * D + CH * g);
#pragma unroll
          for (int k = 0; k < CH / 4; ++k)
            dst[k] = make_float4(o[nt][2 * k][c], o[nt][2 * k][c + 2], o[nt][2 * k + 1][c], o[nt][2 * k + 1][c + 2]);
          if (g == 0)
            *reinterpret_cast<float2*>(p.part_ml + (slot * p.rows_cap + r) * 2) = make_float2(m[nt][c], l[nt][c]);
        }
      }
    // ---- the next segment ----
    u += seg;
    i0 = -kStartUnits;
    if (u < u1 && ++h == heads) {
      h = 0;
      do {
        ++b;
        w = seq_work<MODE>(a, b);
      } while (w.units == 0 && b + 1 < a.s.batch);
      if (w.units == 0) break;   // not with lengths that hold still during the call
    }
  }
}

// Few or short items: a CTA or a cluster of CTAs per item, the item's units
// divided among all their warps, the parts joined in shared memory, then across
// the cluster's.  No scan of the batch, no workspace, one launch: what counts
// there is the latency of one pass.
template <int D, int NT, int W, int MODE>
__global__ void __launch_bounds__(W * 32, 1)
    decode_item_kernel(const __grid_constant__ DecodeArgs p, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v) {
  using C = DecCfg<D, W>;
  constexpr int CH = D / 8, R = NT * 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 ml_s[W][R];
  __shared__ float2 cta_ml[R];
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Ring rg{ptx::smem_u32(smem) + (uint32_t)(wid * C::kStages * C::kStage),
          ptx::smem_u32(smem) + (uint32_t)(C::kBar + wid * C::kStages * 8), 0, 0u};
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) ptx::mbar_init(rg.bars + 8 * i, 1);
    ptx::fence_mbar_init();
  }
  __syncwarp();
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  // CTAs of a cluster are neighbours in the grid
  const unsigned ctas = (unsigned)p.cluster, rank = blockIdx.x % ctas, item = blockIdx.x / ctas;
  const int b = (int)(item / (unsigned)a.p.heads), h = (int)(item % (unsigned)a.p.heads);
  const SeqWork w = seq_work<MODE>(a, b);
  const int rows = w.n * a.group;
  const long long parts = (long long)ctas * W;
  auto begin = [&](int warp) { return (int)((long long)w.units * ((int)rank * W + warp) / parts); };
  const int i0 = begin(wid), i1 = rows > 0 ? begin(wid + 1) : i0;
  float o[NT][D / 16][4], m[NT][2], l[NT][2];
  bool ok = true;
  if (i1 > i0) ok = decode_segment<D, NT, W, MODE>(a, map_k, map_v, rg, b, h, w, i0, i1 - i0, o, m, l);
  // a warp without units, or whose copies did not come, has no part (its
  // weights are zero)
  const bool part_of = i1 > i0 && ok;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (g == 0)
        ml_s[wid][nt * 8 + 2 * t + c] = part_of ? make_float2(m[nt][c], l[nt][c]) : make_float2(-CUDART_INF_F, 0.f);
  __syncthreads();   // no copy of any warp is in flight now: the rings are free
  float* part = reinterpret_cast<float*>(smem);   // [warp][row][D], then [row][D] of the CTA
  float* cta_o = part + W * R * D;
  if (part_of) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = nt * 8 + 2 * t + c;
        if (r >= rows) continue;
        float4* dst = reinterpret_cast<float4*>(part + (wid * R + r) * D + CH * g);
#pragma unroll
        for (int k = 0; k < CH / 4; ++k)
          dst[k] = make_float4(o[nt][2 * k][c], o[nt][2 * k][c + 2], o[nt][2 * k + 1][c], o[nt][2 * k + 1][c + 2]);
      }
  }
  __syncthreads();
  auto store = [&](int r, const float (&v)[D / 32], float top, float ls) {
    const long long row = (long long)(w.r0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
    if (!KVQ_IN_BOUNDS(row, (long long)a.s.rows * a.q_heads, a.status, a.bounds_site)) return;
    const float f = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll
    for (int c = 0; c < D / 32; c += 2) {
      const __nv_bfloat162 z = __floats2bfloat162_rn(v[c] * f, v[c + 1] * f);
      *reinterpret_cast<uint32_t*>(a.out + row * D + (D / 32) * lane + c) = *reinterpret_cast<const uint32_t*>(&z);
    }
    if (lane == 0 && a.lse != nullptr)
      a.lse[row] = (ls == 0.f ? -CUDART_INF_F : 0.6931471805599453f * (top + log2f(ls))) + row_bias<MODE>(a, w, b, h, r);
  };
  // a warp per row, the parts in order.  A part is weighed by 2^(m - M) in two
  // equal factors: far below the others in weight, it may still lead the
  // output by its V scales, up to 2^120, where one factor would be zero
  for (int r = wid; r < rows; r += W) {
    float top = -CUDART_INF_F;
#pragma unroll
    for (int k = 0; k < W; ++k) top = fmaxf(top, ml_s[k][r].x);
    const float base = top > -CUDART_INF_F ? top : 0.f;
    float ls = 0.f, v[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 ml = ml_s[k][r];
      if (ml.y == 0.f) continue;   // nothing there, not even numbers
      const float f = ptx::ex2_approx(0.5f * (ml.x - base));
      ls = fmaf(ml.y * f, f, ls);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) v[c] = fmaf(part[(k * R + r) * D + (D / 32) * lane + c] * f, f, v[c]);
    }
    if (ctas == 1) {
      store(r, v, top, ls);
    } else {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) cta_o[r * D + (D / 32) * lane + c] = v[c];
      if (lane == 0) cta_ml[r] = make_float2(top, ls);
    }
  }
  if (ctas == 1) return;
  ptx::cluster_sync();
  // every CTA of the cluster is here, with or without units: a row is joined
  // by one warp of one CTA, the CTAs' parts in order
  for (int r = (int)rank + (int)ctas * wid; r < rows; r += (int)ctas * W) {
    const uint32_t at_ml = ptx::smem_u32(&cta_ml[r]), at_o = ptx::smem_u32(cta_o + r * D + (D / 32) * lane);
    float top = -CUDART_INF_F;
    for (unsigned k = 0; k < ctas; ++k) top = fmaxf(top, ptx::ld_cluster_f32(ptx::mapa(at_ml, k)));
    const float base = top > -CUDART_INF_F ? top : 0.f;
    float ls = 0.f, v[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) v[c] = 0.f;
    for (unsigned k = 0; k < ctas; ++k) {
      const uint32_t ml = ptx::mapa(at_ml, k), from = ptx::mapa(at_o, k);
      const float f = ptx::ex2_approx(0.5f * (ptx::ld_cluster_f32(ml) - base));
      ls = fmaf(ptx::ld_cluster_f32(ml + 4) * f, f, ls);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) v[c] = fmaf(ptx::ld_cluster_f32(from + 4 * c) * f, f, v[c]);
    }
    store(r, v, top, ls);
  }
  ptx::cluster_sync();   // nobody leaves while its shared memory is read
}

// Joins the parts of items that several warps covered: one block per row of a
// (sequence, cache head), the largest maximum, then sums weighted by
// 2^(m - M) (as two factors), the parts in order.  The block's warps take every fourth part, 32
// lanes hold the channels.
constexpr int kJoinWarps = 4;
template <int D, int MODE>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ DecodeArgs p) {
  constexpr int C = D / 32;
  __shared__ float sum_o[kJoinWarps][D];
  __shared__ float sum_l[kJoinWarps], top_m[kJoinWarps];
  ptx::grid_dependency_wait();
  const PagedAttnArgs& a = p.a;
  const int heads = a.p.heads, cap = a.max_q * a.group;
  const int r = (int)(blockIdx.x % (unsigned)cap);
  const unsigned bh = blockIdx.x / (unsigned)cap;
  const int b = (int)(bh / (unsigned)heads), h = (int)(bh % (unsigned)heads);
  int r0, n;
  seq_rows(a.s, b, r0, n, a.status);
  n = min(n, a.max_q);
  if (r >= n * a.group) return;
  const long long s0 = p.pre[b], span = (p.pre[b + 1] - s0) / heads, total = p.pre[a.s.batch];
  const long long per = max((total + p.warps - 1) / p.warps, (long long)kMinUnits);
  const long long first = s0 + h * span + kStartUnits;
  const long long wa = first / per, wb = (first + span - kStartUnits - 1) / per;
  if (wa == wb) return;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto slot = [&](long long w) { return (2 * w + (w == wa && first > wa * per ? 1 : 0)) * p.rows_cap + r; };
  float top = -CUDART_INF_F;
  for (long long w = wa + threadIdx.x; w <= wb; w += kJoinWarps * 32) top = fmaxf(top, p.part_ml[slot(w) * 2]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  if (lane == 0) top_m[wid] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, top_m[k]);
  const float base = top > -CUDART_INF_F ? top : 0.f;
  float o[C], ls = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll 4
  for (long long w = wa + wid; w <= wb; w += kJoinWarps) {
    const long long at = slot(w);
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
    const float f = ptx::ex2_approx(0.5f * (ml.x - base));
    ls = fmaf(ml.y * f, f, ls);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(p.part_o[at * D + lane + 32 * c] * f, f, o[c]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) sum_o[wid][lane + 32 * c] = o[c];
  if (lane == 0) sum_l[wid] = ls;
  __syncthreads();
  ls = 0.f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) ls += sum_l[k];
  const long long row = (long long)(r0 + r / a.group) * a.q_heads + h * a.group + r % a.group;
  if (!KVQ_IN_BOUNDS(row, (long long)a.s.rows * a.q_heads, a.status, a.bounds_site)) return;
  for (int c = threadIdx.x; c < D; c += kJoinWarps * 32) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) v += sum_o[k][c];
    const __nv_bfloat16 z = __float2bfloat16_rn(ls == 0.f ? 0.f : v / ls);
    a.out[row * D + c] = *reinterpret_cast<const uint16_t*>(&z);
  }
  if (threadIdx.x == 0 && a.lse != nullptr) {
    SeqWork w{};
    w.r0 = r0;
    w.n = n;
    if (MODE != kPlain) w.len = seq_len(a.s, b, a.p.shift, a.status);
    a.lse[row] = (ls == 0.f ? -CUDART_INF_F : 0.6931471805599453f * (top + log2f(ls))) + row_bias<MODE>(a, w, b, h, r);
  }
}

}  // namespace
}  // namespace kvq
