// Attention over the paged cache for many query rows per sequence: prompts,
// chunks, batches of proposed tokens.
//
// Per (sequence, cache head) the rows of its query heads are packed, row r =
// token r / group, head r % group, and a CTA takes 128 NQ of them over all
// their keys, 128 at a time: S = c Q K^T, O += P V with the running base and
// sum of the softmax.  4 d flops per row and key against 2 d bytes per key and
// CTA: at 128 channels bound by the tensor cores.  Measured (24 heads of 128
// channels, 4680 rows, 23400 keys): 0.98 ms, 1380 TFLOP/s, with other inputs in
// each call, 0.945 ms on the same ones again and again: 3400 cycles a tile of
// 128 keys and 256 rows, of which the products take 2048 at their nominal rates.
// They do not reach them: Q K^T reads both operands from shared memory, all of
// its 128 bytes a cycle, and every commit and every instruction of the issuing
// thread shows (four commits less a tile 6 %, its loop unrolled by two tiles
// 2 %).  At 64 channels the products are half as long and the softmax is not:
// the tensor pipe is active 34 % of the time, not 56 (1536 rows of 24 heads,
// 8192 keys), 256 rows of 32 sequences of 16384 keys and 8 heads take 375 us.
// Leaving out the exponentials would save 2 %, the conversion of V nothing;
// scores in halves of 64 keys, so that the next ones start earlier, read the
// query twice as often: 1.34 ms.
//
// Products on tcgen05, accumulators in tensor memory.
// - Q K^T: the E4M3 key tile goes from the page by TMA straight to the tensor
//   core (kind::f8f6f4): no conversion, no copy.  The BF16 query row, scaled
//   by a power of two to a largest magnitude in [128, 256), is split into E4M3
//   high and low parts, two contractions at twice the 16-bit rate: 4 + 4 bits
//   hold BF16's 8 exactly for elements down to 2^-9 of the row's largest, and
//   smaller ones to 2^-17 of it.
// - P V: P in FP16 from tensor memory (kind::f16); V codes to FP16 (exact) by
//   four warps, as the transposed operand.  P in two E4M3 parts would spare
//   that, but its range (2^-9 to 448) is too short for softmax weights.
// Page scales are powers of two outside the products: K's on the scores, V's
// (2^ev) on the weight before it is rounded, as an addend to the exponent.  A
// row's base m follows score plus ev over the keys that the row attends to: it
// is raised only when a weight would leave FP16 (64 keys' sum past 2^15), to
// leave the largest at 2^9, so products of a weight and its scale down to 2^-33
// of the row's largest remain, whatever scales other pages have.
// The sum l of weights has the same base but no V scale: each block of 16 keys
// adds its weights' sum times 2^-ev.  The largest score is within 60 of m - 15
// to m - 9 on either side, so l stays inside fp32.
//
// Roles: two groups of 4 warps softmax (one row per thread), 4 warps V
// conversion, one MMA thread, one TMA warp.  With NQ = 2 a group has a query
// tile of its own; the two alternate on the tensor core (PV0 QK0' PV1 QK1'),
// each key tile is read and converted once for 256 rows.  With NQ = 1 (at most
// 128 rows a head) the groups take the key tiles of one query tile in turn,
// each with its own base, sum and O, and join at the end: with one group alone
// 64 rows of 32 sequences, 16384 keys and 8 heads took 440 us, not 261.
#pragma once

#include <math_constants.h>

#include "kvq_checks.cuh"
#include "kvq_pages.cuh"

namespace kvq {
namespace {

constexpr int kTileKeys = 128;
constexpr int kVStages = 2, kMetaSlots = 8;
// a slot of a tile's page scales, per block of 16 keys: 2^e of K [8], V's e [8]
// (as float) and 2^-that [8]; then the mask of blocks whose page is there, and
// 0.0, or kWideMark where the sum of weights needs exponentials of its own
constexpr int kMetaBytes = 128, kMetaShift = 32, kMetaInv = 64, kMetaThere = 96, kMetaWide = 100;
// Weights with V's scale in them flush to zero 126 binades below m, 135 or more
// below the row's largest product.  On a page whose V scale is D binades under
// the largest one so far that leaves out of l what is 135 - D binades or more
// below the largest weight: nothing that 2^30 keys could add up to 2^-15 of, up
// to D = 90.  Past it a tile's sum is taken from the scores alone.  The mark is
// a number beyond every bound, so that the test for a new base takes notice of
// it by itself (a branch of its own cost 1 to 2 %).
constexpr int kWideSpan = 90;
constexpr uint32_t kWideMark = 0x70000000u;   // 1.6e29

template <int D, int NQ>
struct ChunkCfg {
  static constexpr int kKStages = NQ == 2 ? 2 : 3;
  static constexpr int kQT = 128 * D;              // one E4M3 query tile
  static constexpr int kQ = 0;                     // [NQ][high, low]
  static constexpr int kK = NQ * 2 * kQT;          // key codes
  static constexpr int kKT = kTileKeys * D;
  static constexpr int kVr = kK + kKStages * kKT;  // value codes as they arrive
  static constexpr int kV = kVr + kVStages * kKT;  // values in FP16, D / 64 sub-tiles [128][64]
  static constexpr int kVT = 2 * kKT;
  static constexpr int kMeta = kV + kVStages * kVT;
  static constexpr int kBar = kMeta + kMetaSlots * kMetaBytes;
  static constexpr int kBytes = kBar + 512;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr int kSoftmaxWarps = 8;
  static constexpr int kMmaWarp = kSoftmaxWarps + 4;
  static constexpr int kThreads = (kSoftmaxWarps + 6) * 32;
  static constexpr int kTO = 256;                  // O tiles behind two score buffers
  static constexpr int kTCols = 512;
  static_assert(kTO + 2 * D <= kTCols, "tensor memory");
  static_assert(kAlloc <= 232448, "shared memory");
};

// A commit costs the tensor core some of its time (one less a tile: 2 %), so
// nothing is signalled twice.  "Scores of a tile ready" also says that all
// products issued before them are done, which frees a key stage and a value
// stage; there are as many barriers for it as keep their phases apart.
enum : int {
  kCbQ = 0,         // query tiles written (4 NQ arrivals, one per warp)
  kCbFullK = 1,     // [3] key codes landed
  kCbFullVr = 4,    // [2] value codes landed
  kCbEmptyVr = 6,   // [2] value codes read (4 arrivals)
  kCbFullV = 8,     // [2] FP16 values written (4 arrivals)
  kCbS = 10,        // [4] scores ready: tile j of query tile q at 2 q + j % 2
                    // (NQ = 2), tile j at j % 4 (NQ = 1)
  kCbP = 14,        // [2] weights of keys 0-63 written, O rescaled (4 arrivals)
  kCbPb = 16,       // [2] weights of keys 64-127 written (4 arrivals)
  kCbHalf = 18,     // [2] PV of keys 0-63 done, when a softmax warp asked
  kCbODone = 20,    // every MMA done
  kCbMeta = 21,     // [8] a tile's page exponents written.  Not the key
                    // barrier: its stage can be refilled, and its phase
                    // passed twice, before a slow softmax warp looks at it
  kCbCount = 29
};

struct ChunkArgs {
  PagedAttnArgs a;
  int q_tiles;        // row tiles of 128 NQ per (sequence, cache head), at most
  int splits;         // key ranges per row tile
  float* part_o;      // [splits][rows * q_heads][D] (splits > 1)
  float* part_ml;     // [splits][rows * q_heads][2]
};

// the page of a block of 16 keys: id (-1: none), scale exponents
struct BlockPage {
  int id, ek, ev;
};

// shared memory by its 32-bit address (a generic pointer would make each
// access a generic one)
__device__ __forceinline__ uint4 lds_u4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds_u2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void sts_u4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts_u2(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

// where the base of a row starts: every weight against it is infinite
constexpr float kLowest = -1e30f;

// log of a sum l of weights against base m (binades).  l can be far from 1, so
// its exponent joins m before its logarithm does: both terms then have the
// size of the result.
__device__ __forceinline__ float lse_of(float m, float l) {
  if (l == 0.f) return -CUDART_INF_F;
  const int r = min(max((int)(__float_as_uint(l) >> 23) - 127, -126), 126);
  return 0.6931471805599453f * ((m + (float)r) + log2f(l * pow2f(-r)));
}

// weights of 16 scores, 2^(score scale + shift), as FP16 pairs, and their sum
__device__ __forceinline__ void exp_block(const uint32_t* s, float scale, float shift, uint32_t* pk, float& sum) {
  const uint64_t s2 = ptx::f2_pack(scale, scale), b2 = ptx::f2_pack(shift, shift);
  uint64_t acc = ptx::f2_pack(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float x0, x1;
    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), s2, b2),
                   x0, x1);
    const float e0 = ptx::ex2_approx(x0), e1 = ptx::ex2_approx(x1);
    acc = ptx::f2_add(acc, ptx::f2_pack(e0, e1));
    pk[k] = ptx::f16x2_rn(e0, e1);
  }
  float x, y;
  ptx::f2_unpack(acc, x, y);
  sum = x + y;
}
// scores of columns outside [lo, hi) become -inf
__device__ __forceinline__ void mask_block(uint32_t* s, int lo, int hi) {
#pragma unroll
  for (int k = 0; k < 16; ++k) s[k] = k >= lo && k < hi ? s[k] : 0xff800000u;
}


// A score with its V exponent, each step rounded by itself: its distance from a
// base taken from such a sum is what it says, however large the scores.  (A
// fused product's distance holds what the base's rounding left out, 2^16 binades
// at a score of 2^40: the weights of the largest keys would be zero or infinite.)
__device__ __forceinline__ float with_ev(float s, float ck, float ev) { return __fadd_rn(__fmul_rn(s, ck), ev); }
constexpr float kFarBase = 1048576.f;   // a base that large, 2^20 binades, takes with_ev's distances
// 64 weights by with_ev's distances, written over the scores, and their sum from
// exponents without V's.  Out of line, so that it takes no place among the
// instructions of ordinary tiles (in line 2 to 4 %).
__device__ __noinline__ float weights_apart(uint32_t t_h, uint32_t mh, float cq, float m, int lo, int hi,
                                            uint32_t there) {
  float sum = 0.f;
#pragma unroll 1
  for (int k = 0; k < 4; k += 2) {
    uint32_t v[32], w[16];
    ptx::tmem_ld32(t_h + 16 * k, v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float ck = fmaxf(cq * lds_f(mh + 4 * (k + i)), 1.2e-38f), ev = lds_f(mh + kMetaShift + 4 * (k + i));
      mask_block(v + 16 * i, (there >> (k + i)) & 1u ? lo - 16 * (k + i) : 16, hi - 16 * (k + i));
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x0 = with_ev(__uint_as_float(v[16 * i + 2 * c]), ck, ev) - m;
        const float x1 = with_ev(__uint_as_float(v[16 * i + 2 * c + 1]), ck, ev) - m;
        w[8 * i + c] = ptx::f16x2_rn(ptx::ex2_approx(x0), ptx::ex2_approx(x1));
        sum += ptx::ex2_approx(x0 - ev) + ptx::ex2_approx(x1 - ev);
      }
    }
    ptx::tmem_st16(t_h + 8 * k, w);   // (columns that the loads are past)
  }
  ptx::tmem_st_wait();
  return sum;
}

// words that pass between a softmax warp and the MMA thread
__device__ __forceinline__ void st_release(uint32_t at, uint32_t v) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire(uint32_t at) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
// waits until the word is v, bounded
__device__ __noinline__ bool wait_word(uint32_t at, uint32_t v, unsigned long long limit_ns, volatile int* abort,
                                       int* status) {
  const uint64_t t0 = ptx::globaltimer();
  while (ld_acquire(at) != v) {
    if (*abort) return false;
    if (ptx::globaltimer() - t0 > limit_ns) {
      *abort = 1;
      atomicCAS(status, 0, (int)KVQ_ERR_TIMEOUT);
      return false;
    }
    __nanosleep(100);
  }
  return true;
}

// one arrival for a warp whose lanes are all done (a barrier takes its
// arrivals one after another: 128 of them cost some hundred cycles)
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

template <int D, int NQ>
__global__ void __launch_bounds__(ChunkCfg<D, NQ>::kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkArgs p, const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v) {
  using C = ChunkCfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const PagedAttnArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();

  // the longest row tiles (the last ones, under a causal mask) go first
  const int heads = a.p.heads;
  unsigned at = blockIdx.x;
  const int h = (int)(at % (unsigned)heads);
  at /= (unsigned)heads;
  const int b = (int)(at % (unsigned)a.s.batch);
  at /= (unsigned)a.s.batch;
  const int split = (int)(at % (unsigned)p.splits);
  const int qt = p.q_tiles - 1 - (int)(at / (unsigned)p.splits);
  int r0, n;
  seq_rows(a.s, b, r0, n, a.status);
  if (n > a.max_q) {
    page_error(a.status);
    n = a.max_q;
  }
  const int rows = n * a.group;                 // of this head
  const int row0 = qt * (128 * NQ);
  if (row0 >= rows) return;
  const int len = seq_len(a.s, b, a.p.shift, a.status);
  const int t0 = len - n;                       // position of row 0
  // keys that some row of the tile attends to, and their 128-key tiles
  const int i_first = row0 / a.group, i_last = (min(rows, row0 + 128 * NQ) - 1) / a.group;
  const int key_hi = a.causal ? max(min(len, t0 + i_last + 1), 0) : len;
  const int key_lo = a.window > 0 ? max(0, t0 + i_first - a.window + 1) : 0;
  const int tile_lo = key_lo / kTileKeys;
  const int tiles = key_hi > key_lo ? (key_hi + kTileKeys - 1) / kTileKeys - tile_lo : 0;
  const int j0 = (int)((long long)tiles * split / p.splits), j1 = (int)((long long)tiles * (split + 1) / p.splits);
  const int n_t = j1 - j0;
  const int base = (tile_lo + j0) * kTileKeys;  // first key of local tile 0

  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kBar + kCbCount * 8);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBar + kCbCount * 8 + 4);
  // per group: the tile (+ 1) whose first half's product a softmax warp waits
  // for, and the last one it was told of.  It needs that only when its base
  // rises within a tile, too rarely for a commit in every tile (3 %).
  const uint32_t ask0 = ptx::smem_u32(smem + C::kBar + kCbCount * 8 + 8), told0 = ask0 + 8;
  const uint32_t bar0 = ptx::smem_u32(smem + C::kBar);
  auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  if (tid == 0) {
    ptx::mbar_init(BAR(kCbQ), 4 * NQ);
    for (int i = 0; i < C::kKStages; ++i) ptx::mbar_init(BAR(kCbFullK + i), 1);
    for (int i = 0; i < 4; ++i) ptx::mbar_init(BAR(kCbS + i), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(BAR(kCbFullVr + i), 1);
      ptx::mbar_init(BAR(kCbEmptyVr + i), 4);
      ptx::mbar_init(BAR(kCbFullV + i), 4);
      ptx::mbar_init(BAR(kCbP + i), 4);
      ptx::mbar_init(BAR(kCbPb + i), 4);
      ptx::mbar_init(BAR(kCbHalf + i), 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) ptx::mbar_init(BAR(kCbMeta + i), 1);
    ptx::mbar_init(BAR(kCbODone), 1);
    *abort = 0;
    for (int i = 0; i < 2; ++i) {
      st_release(ask0 + 4 * i, 0u);
      st_release(told0 + 4 * i, 0u);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::kTCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const unsigned long long lim = a.wait_limit_ns;
  const uint32_t sm = ptx::smem_u32(smem);
  // barrier and phase of tile j's scores (query tile q)
  auto s_bar = [](int q, int j) { return kCbS + (NQ == 2 ? 2 * q + (j & 1) : (j & 3)); };
  auto s_par = [](int j) { return (uint32_t)(NQ == 2 ? j >> 1 : j >> 2) & 1u; };

  if (warp < C::kSoftmaxWarps) {
    // =========================== softmax ===========================
    const int q = warp >> 2;
    const int r = (warp & 3) * 32 + lane;        // TMEM lane, row of the query tile
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // row of the head's rows; one past the last repeats it and is not stored
    const int qoff = row0 + (NQ == 2 ? q * 128 : 0);
    const bool live = qoff + r < rows;
    const int row = min(qoff + r, rows - 1);
    const int tok = row / a.group;
    const int hq = h * a.group + row % a.group;
    // a warp without a row of its own only keeps the barriers going: its
    // lanes of the products go nowhere
    const bool idle = qoff + (warp & 3) * 32 >= rows;
    // ---- the query row: scale, split, store (K-major, swizzled) ----
    float cq;
    {
      uint4 raw[D / 8];
      const uint4* qp = reinterpret_cast<const uint4*>(a.q + (long long)(r0 + tok) * a.q_row_stride +
                                                       (long long)hq * a.q_head_stride);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) raw[c] = __ldg(qp + c);
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = max(mx, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
      }
      const int e = max((int)(mx >> 7), 1) - 127 - 7;      // largest magnitude to [2^7, 2^8)
      // (an infinity or a NaN makes the whole row NaN)
      const float f0 = mx < 0x7f80u ? pow2f(-(e / 2)) : CUDART_NAN_F, f1 = pow2f(-(e - e / 2));
      cq = a.scale * 1.4426950408889634f * pow2f(e / 2) * pow2f(e - e / 2);
      const uint32_t hi_t = sm + C::kQ + (NQ == 2 ? q : 0) * 2 * C::kQT;
      if (NQ == 2 || q == 0) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t wh[4], wl[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4& v = raw[2 * c + (k >> 1)];
            const uint32_t w0 = (k & 1) ? v.z : v.x, w1 = (k & 1) ? v.w : v.y;
            const float x0 = __uint_as_float(w0 << 16) * f0 * f1, x1 = __uint_as_float(w0 & 0xffff0000u) * f0 * f1;
            const float x2 = __uint_as_float(w1 << 16) * f0 * f1, x3 = __uint_as_float(w1 & 0xffff0000u) * f0 * f1;
            wh[k] = e4m3x4(x0, x1, x2, x3);
            const uint32_t h01 = f16x2_of_e4m3x2((uint16_t)wh[k]), h23 = f16x2_of_e4m3x2((uint16_t)(wh[k] >> 16));
            const float2 a01 = __half22float2(*reinterpret_cast<const __half2*>(&h01));
            const float2 a23 = __half22float2(*reinterpret_cast<const __half2*>(&h23));
            wl[k] = e4m3x4(x0 - a01.x, x1 - a01.y, x2 - a23.x, x3 - a23.y);
          }
          const int off = D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
          sts_u4(hi_t + off, make_uint4(wh[0], wh[1], wh[2], wh[3]));
          sts_u4(hi_t + C::kQT + off, make_uint4(wl[0], wl[1], wl[2], wl[3]));
        }
        ptx::fence_proxy_async_smem();
        warp_arrive(BAR(kCbQ));
      }
    }

    // keys this row attends to, from the first key of local tile 0
    const int tq = t0 + tok;
    const int hi_r = (a.causal ? min(len, tq + 1) : len) - base;
    const int lo_r = (a.window > 0 ? max(0, tq - a.window + 1) : 0) - base;
    float m = kLowest, l = 0.f;
    const uint32_t t_o = tmem + C::kTO + q * D + lane_off;
    bool ok = true;
    const uint32_t t_s = tmem + q * 128 + lane_off;
    for (int j = NQ == 2 ? 0 : q; j < n_t; j += NQ == 2 ? 1 : 2) {
      const bool first = NQ == 2 ? j == 0 : j < 2;
      // a slot of scales is written again 8 tiles later, the TMA warp at most
      // 5 ahead of the softmax (key stages and score buffers)
      ok = page_wait(BAR(kCbMeta + (j & (kMetaSlots - 1))), (j / kMetaSlots) & 1, lim, abort, a.status) &&
           page_wait(BAR(s_bar(q, j)), s_par(j), lim, abort, a.status);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      if (idle) {
        warp_arrive(BAR(kCbP + q));
        warp_arrive(BAR(kCbPb + q));
        continue;
      }
      const uint32_t mt = sm + C::kMeta + (j & (kMetaSlots - 1)) * kMetaBytes;
      const uint32_t there = lds_u(mt + kMetaThere);
      const int at0 = j * kTileKeys;
      const bool whole = __all_sync(0xffffffffu, there == 255u && lo_r <= at0 && hi_r >= at0 + kTileKeys);
      auto rescale_o = [&](float f) {
        const uint64_t f2 = ptx::f2_pack(f, f);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[16];
          ptx::tmem_ld16(t_o + 16 * c, v);
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float x, y;
            ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), f2), x, y);
            v[k] = __float_as_uint(x);
            v[k + 1] = __float_as_uint(y);
          }
          ptx::tmem_st16(t_o + 16 * c, v);
        }
      };
      // ---- weights, 64 keys at a time.  Those of keys 0-63 are handed over
      // as soon as they are there, so that their product runs beside the
      // rest.  The loop stays a loop: a body that fits the instruction
      // buffers, its scores in the registers they were loaded to ----
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t t_h = t_s + 64 * half, mh = mt + 16 * half;
        uint32_t pk[2][16];
        float hat, sum;
        const float wide = lds_f(mt + kMetaWide);
        auto scores = [&](uint32_t (&cur)[64]) {
          ptx::tmem_ld64(t_h, cur);
          if (!whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int at = at0 + 64 * half + 16 * k;
              mask_block(cur + 16 * k, (there >> (4 * half + k)) & 1u ? lo_r - at : 16, hi_r - at);
            }
          }
        };
        auto weights = [&](const uint32_t (&cur)[64]) {
          hat = wide;
          sum = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // (a scale that underflows must not meet the -inf of a masked score)
            const float ck = fmaxf(cq * lds_f(mh + 4 * k), 1.2e-38f);
            float b;
            exp_block(cur + 16 * k, ck, lds_f(mh + kMetaShift + 4 * k) - m, pk[k >> 1] + 8 * (k & 1), b);
            hat += b;
            sum = fmaf(b, lds_f(mh + kMetaInv + 4 * k), sum);
          }
        };
        {
          uint32_t cur[64];
          scores(cur);
          weights(cur);
        }
        // past FP16 (or the first weights of all, against the lowest base): a
        // new base, and what there is so far follows it
        if (__builtin_expect(__any_sync(0xffffffffu, hat > 32768.0f), 0)) {
          uint32_t cur[64];
          scores(cur);
          float top = kLowest;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float most = -CUDART_INF_F;
#pragma unroll
            for (int i = 0; i < 16; ++i) most = fmaxf(most, __uint_as_float(cur[16 * k + i]));
            top = fmaxf(top, with_ev(most, fmaxf(cq * lds_f(mh + 4 * k), 1.2e-38f), lds_f(mh + kMetaShift + 4 * k)));
          }
          // (by two factors: l may stand 75 binades above 2^m)
          const float m_new = fmaxf(m, __fadd_ru(top, -9.f)), f = exp2f(0.5f * (m - m_new));
          m = m_new;
          l = l * f * f;
          weights(cur);
          if (__any_sync(0xffffffffu, wide != 0.f || (fabsf(m) > kFarBase && m > kLowest))) {
            sum = weights_apart(t_h, mh, cq, m, lo_r - at0 - 64 * half, hi_r - at0 - 64 * half, there >> (4 * half));
            ptx::tmem_ld16(t_h, pk[0]);
            ptx::tmem_ld16(t_h + 16, pk[1]);
          }
          if (__any_sync(0xffffffffu, f != 1.f)) {
            // (the product of the first half is still under way; the group's
            // previous tile's was done before these scores were)
            if (half == 1) {
              if (lane == 0) st_release(ask0 + 4 * q, (uint32_t)j + 1u);
              ok = __all_sync(0xffffffffu, ok && wait_word(told0 + 4 * q, (uint32_t)j + 1u, lim, abort, a.status));
            }
            ptx::tc_fence_after();
            if (!first || half == 1) rescale_o(f * f);
          }
        }
        l += sum;
        // over the first 32 of the 64 score columns just read
        ptx::tmem_st16(t_h, pk[0]);
        ptx::tmem_st16(t_h + 16, pk[1]);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        warp_arrive(BAR((half == 0 ? kCbP : kCbPb) + q));
      }
      if (!ok) break;
    }

    // ---- result ----
    if (ok) ok = page_wait(BAR(kCbODone), 0, lim, abort, a.status);
    ok = __all_sync(0xffffffffu, ok && !*abort);
    ptx::tc_fence_after();
    // NQ = 1: the second group's share goes through shared memory, whose tiles
    // nobody reads any more
    const bool mine = n_t > (NQ == 2 ? 0 : q);   // the group had tiles
    float f0 = 1.f, f1 = 0.f;
    const uint32_t part_at = sm + C::kV + 4 * r, ml_at = sm + C::kK + 8 * r;
    if constexpr (NQ == 1) {
      if (q == 1) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (!(mine && ok)) break;
          ptx::tmem_ld32(t_o + 32 * c, v);
#pragma unroll
          for (int k = 0; k < 32; ++k) sts_f(part_at + (32 * c + k) * 512, __uint_as_float(v[k]));
        }
        sts_u2(ml_at, __float_as_uint(m), __float_as_uint(mine && ok ? l : 0.f));
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");   // the eight softmax warps
      if (q == 0) {
        const uint2 ml = lds_u2(ml_at);
        const float m1 = __uint_as_float(ml.x), l1 = __uint_as_float(ml.y), top = fmaxf(m, m1);
        const float h0 = exp2f(0.5f * (m - top)), h1 = l1 == 0.f ? 0.f : exp2f(0.5f * (m1 - top));
        l = l * h0 * h0 + l1 * h1 * h1;   // (by two factors, as above)
        f0 = h0 * h0;
        f1 = h1 * h1;
        m = top;
      }
    }
    if (ok && (NQ == 2 || q == 0)) {
      const long long orow = (long long)(r0 + tok) * a.q_heads + hq;
      const bool store = live && KVQ_IN_BOUNDS(orow, (long long)a.s.rows * a.q_heads, a.status, a.bounds_site);
      const bool part = p.splits > 1;
      const float f = part ? 1.f : (l == 0.f ? 0.f : 1.f / l);
      f0 *= f;
      f1 *= f;
      const long long prow = (long long)split * a.s.rows * a.q_heads + orow;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        if (mine) {
          ptx::tmem_ld32(t_o + 32 * c, v);   // warp-collective: every lane
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float x = __uint_as_float(v[k]) * f0;
          if (NQ == 1 && f1 != 0.f) x = fmaf(lds_f(part_at + (32 * c + k) * 512), f1, x);
          v[k] = __float_as_uint(x);
        }
        if (!store) continue;
        if (part) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                 __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
        } else {
          uint4* dst = reinterpret_cast<uint4*>(a.out + orow * D + 32 * c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * i]),
                                                             __uint_as_float(v[8 * k + 2 * i + 1]));
              z[i] = *reinterpret_cast<const uint32_t*>(&y);
            }
            dst[k] = make_uint4(z[0], z[1], z[2], z[3]);
          }
        }
      }
      if (store) {
        if (part) *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m, l);
        else if (a.lse != nullptr) a.lse[orow] = lse_of(m, l);
      }
    }
  } else if (warp < C::kMmaWarp) {
    // ====================== values to FP16 ======================
    const int r = tid - C::kSoftmaxWarps * 32;   // key of the tile
    // what no row attends to must not reach the product (zero times NaN)
    const int first = a.window > 0 ? max(0, t0 - a.window + 1) : 0;
    for (int j = 0; j < n_t; ++j) {
      const int s = j & 1;
      const uint32_t par = (j >> 1) & 1;
      if (!page_wait(BAR(kCbFullVr + s), par, lim, abort, a.status)) break;
      const int key = base + j * kTileKeys + r;
      const uint32_t there = lds_u(sm + C::kMeta + (j & (kMetaSlots - 1)) * kMetaBytes + kMetaThere);
      const bool use = key >= first && key < len && ((there >> (r >> 4)) & 1u);
      uint4 raw[D / 16];
      const uint32_t src = sm + C::kVr + s * C::kKT;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int off = D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
        raw[c] = lds_u4(src + off);
        if (!use) raw[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      warp_arrive(BAR(kCbEmptyVr + s));
      // PV of tile j - 2 is done with this stage: it was issued before the
      // scores of tile j - 1 of the second query tile (NQ = 1: of tile j)
      if (j >= 2) {
        const int after = NQ == 2 ? j - 1 : j;
        if (!page_wait(BAR(s_bar(1, after)), s_par(after), lim, abort, a.status)) break;
      }
      const uint32_t dst = sm + C::kV + s * C::kVT;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ch = 2 * c + i;               // 16-byte chunk: channels 8 ch ..
          uint4 o;
          o.x = f16x2_of_e4m3x2((uint16_t)w[2 * i]);
          o.y = f16x2_of_e4m3x2((uint16_t)(w[2 * i] >> 16));
          o.z = f16x2_of_e4m3x2((uint16_t)w[2 * i + 1]);
          o.w = f16x2_of_e4m3x2((uint16_t)(w[2 * i + 1] >> 16));
          sts_u4(dst + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4), o);
        }
      }
      ptx::fence_proxy_async_smem();
      warp_arrive(BAR(kCbFullV + s));
    }
  } else {
    if (warp == C::kMmaWarp) {
    // ============================= MMA =============================
    if (lane == 0) {
      constexpr uint32_t kIdS = ptx::idesc_f8kind(128, kTileKeys);
      constexpr uint32_t kIdO = ptx::idesc_f16kind(128, D, true, false);
      constexpr uint32_t kLay = D == 128 ? ptx::kLayoutSw128 : ptx::kLayoutSw64;
      const uint32_t s_base = sm;
      const uint64_t d8 = ptx::smem_desc(s_base, 16, 8 * D, kLay);       // E4M3 rows of D bytes
      const uint64_t dv = ptx::smem_desc(s_base, 16384, 1024, ptx::kLayoutSw128);
      auto plus = [](uint64_t d, uint32_t off) { return d + (uint64_t)(off >> 4); };
      bool ok = n_t == 0 || page_wait(BAR(kCbQ), 0, lim, abort, a.status);
      auto qk = [&](int ks, int q, uint32_t dst) {
        const uint64_t db = plus(d8, C::kK + ks * C::kKT);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint64_t da = plus(d8, C::kQ + (2 * q + part) * C::kQT);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            ptx::mma_f8(dst, da + (uint64_t)(2 * k), db + (uint64_t)(2 * k), kIdS, (part > 0 || k > 0) ? 1u : 0u);
        }
      };
      auto pv = [&](int j, int vs, int q, int half, uint32_t p_tmem) {
        const uint64_t db = plus(dv, C::kV + vs * C::kVT);
#pragma unroll
        for (int k = 0; k < kTileKeys / 32; ++k) {
          // weights of 64 keys: 32 columns, 64 apart
          const int kk = 4 * half + k;
          ptx::mma_f16_ts(tmem + C::kTO + q * D, p_tmem + 64 * half + 8 * k,
                          db + (uint64_t)((kk * 2048) >> 4), kIdO, (j > 2 - NQ || kk > 0) ? 1u : 0u);
        }
      };
      int ks = 0;
      uint32_t kph = 0;
      auto next_k = [&]() {
        const bool good = page_wait(BAR(kCbFullK + ks), kph, lim, abort, a.status);
        ptx::tc_fence_after();
        return good;
      };
      auto step_k = [&]() {
        if (++ks == C::kKStages) {
          ks = 0;
          kph ^= 1u;
        }
      };
      // weights of the second half, or before them the question for the
      // first half's product
      uint32_t half_ph = 0;   // phases of the two barriers
      auto wait_second = [&](int grp, uint32_t par, uint32_t tile) {
        const uint64_t t_0 = ptx::globaltimer();
        while (!ptx::mbar_try_wait_sleep(BAR(kCbPb + grp), par, 1000u)) {
          if (ld_acquire(ask0 + 4 * grp) == tile && ld_acquire(told0 + 4 * grp) != tile) {
            ptx::mma_commit(BAR(kCbHalf + grp));
            if (!page_wait(BAR(kCbHalf + grp), (half_ph >> grp) & 1u, lim, abort, a.status)) return false;
            half_ph ^= 1u << grp;
            ptx::tc_fence_before();
            st_release(told0 + 4 * grp, tile);
          }
          if (*abort) return false;
          if (ptx::globaltimer() - t_0 > lim) {
            *abort = 1;
            atomicCAS(a.status, 0, (int)KVQ_ERR_TIMEOUT);
            return false;
          }
        }
        return true;
      };
      if (ok && n_t > 0) {
        ptx::tc_fence_after();
        ok = next_k();
        if (ok) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            qk(ks, q, tmem + q * 128);
            ptx::mma_commit(BAR(s_bar(q, 0)));
          }
          step_k();
        }
        // two tiles a turn: stages and barriers that alternate are constants
        // then (the issue of one group's products waits behind this thread)
        for (int j0 = 0; j0 < n_t && ok; j0 += 2) {
          const uint32_t ph = (uint32_t)(j0 >> 1) & 1u;   // of what alternates by tiles
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int j = j0 + u;
            if (!ok || j >= n_t) break;
            const bool more = j + 1 < n_t;
            if (NQ == 1 && more) {
              if (!(ok = next_k())) break;
              qk(ks, 0, tmem + ((u + 1) & 1) * 128);
              ptx::mma_commit(BAR(s_bar(0, j + 1)));
              step_k();
            }
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              if (!ok) break;
              const int grp = NQ == 2 ? q : u;
              const uint32_t par = NQ == 2 ? (uint32_t)u : ph, t_p = tmem + grp * 128;
              if (!(ok = page_wait(BAR(kCbP + grp), par, lim, abort, a.status))) break;
              if (q == 0 && !(ok = page_wait(BAR(kCbFullV + u), ph, lim, abort, a.status))) break;
              ptx::tc_fence_after();
              pv(j, u, grp, 0, t_p);
              if (!ptx::mbar_try_wait_sleep(BAR(kCbPb + grp), par, 2000u) &&
                  !(ok = wait_second(grp, par, (uint32_t)j + 1u)))
                break;
              ptx::tc_fence_after();
              pv(j, u, grp, 1, t_p);
              if (NQ == 2 && more) {
                const int kst = (u + 1) & 1;
                if (q == 0) {
                  if (!(ok = page_wait(BAR(kCbFullK + kst), ph ^ (uint32_t)u, lim, abort, a.status))) break;
                  ptx::tc_fence_after();
                }
                qk(kst, q, tmem + q * 128);
                ptx::mma_commit(BAR(kCbS + 2 * q + kst));
              }
            }
          }
        }
      }
      // every MMA issued is done before the tensor memory goes back
      ptx::mma_commit(BAR(kCbODone));
      page_drain(BAR(kCbODone), 0, lim);
    }
    __syncwarp();
    } else if (warp == C::kMmaWarp + 1) {
    // ============================== TMA ==============================
    const uint32_t s_base = sm;
    // pages of four tiles at a time, lane 8 i + k that of keys [16 k, 16 k +
    // 16) of tile j + i: two dependent loads, issued four tiles ahead of
    // their use (one tile at a time they bound the whole kernel)
    auto look = [&](int j) -> BlockPage {
      BlockPage o{-1, -1000, -1000};
      const int key = base + j * kTileKeys + 16 * lane;
      // (a page wholly before every row's window may be gone already)
      if (j + (lane >> 3) < n_t && key < key_hi && ((long long)((key >> a.p.shift) + 1) << a.p.shift) > key_lo) {
        o.id = seq_page(a.s, b, key >> a.p.shift, a.p.n_pages, a.status);
        if (o.id >= 0) {
          const long long blk = (long long)o.id * heads + h;
          o.ek = scale_exp(__ldg(a.p.scale[0] + blk));
          o.ev = scale_exp(__ldg(a.p.scale[1] + blk));
        }
      }
      return o;
    };
    BlockPage four = look(0), next_four = look(4);
    int ev_top = -1000;   // largest V exponent so far
    int ks = 0, last_k = -1, last_v = -1;
    bool ok = true;
    for (int j = 0; j < n_t; ++j) {
      if (j > 0 && (j & 3) == 0) {
        four = next_four;
        next_four = look(j + 4);
      }
      const int from = 8 * (j & 3) + (lane & 7);
      BlockPage cur;
      cur.id = __shfl_sync(0xffffffffu, four.id, from);
      cur.ek = __shfl_sync(0xffffffffu, four.ek, from);
      cur.ev = __shfl_sync(0xffffffffu, four.ev, from);
      if (lane >= 8) cur.id = -1;
      const bool box = cur.id >= 0 && ((16 * lane) & (a.p.page - 1)) == 0;
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, box));
      const uint32_t bytes = boxes * (uint32_t)(a.p.page * D);
      if (j >= C::kKStages) {   // the scores of the tile before in this stage are ready
        const int before = j - C::kKStages;
        ok = page_wait(BAR(s_bar(NQ - 1, before)), s_par(before), lim, abort, a.status);
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      {
        const uint32_t mt = sm + C::kMeta + (j & (kMetaSlots - 1)) * kMetaBytes;
        ev_top = max(ev_top, (int)__reduce_max_sync(0xffffffffu, cur.id >= 0 ? cur.ev : -1000));
        const int ev_low = (int)__reduce_min_sync(0xffffffffu, cur.id >= 0 ? cur.ev : 1000);
        const uint32_t there = __ballot_sync(0xffffffffu, cur.id >= 0);
        if (lane < 8) {
          const int ev = cur.id >= 0 ? cur.ev : 0;
          sts_f(mt + 4 * lane, cur.id >= 0 ? pow2f(cur.ek) : 1.f);
          sts_f(mt + kMetaShift + 4 * lane, (float)ev);
          sts_f(mt + kMetaInv + 4 * lane, pow2f(-ev));
        }
        if (lane == 0) sts_u2(mt + kMetaThere, there, ev_top - ev_low > kWideSpan ? kWideMark : 0u);
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(BAR(kCbMeta + (j & (kMetaSlots - 1))));
        if (bytes > 0) ptx::mbar_expect_tx(BAR(kCbFullK + ks), bytes); else ptx::mbar_arrive(BAR(kCbFullK + ks));
      }
      __syncwarp();
      if (box)
        ptx::tma_load_3d(s_base + C::kK + ks * C::kKT + 16 * lane * D, &map_k, 0, 0, cur.id * heads + h, BAR(kCbFullK + ks));
      last_k = j;
      if (j >= kVStages) ok = page_wait(BAR(kCbEmptyVr + (j & 1)), ((j >> 1) - 1) & 1, lim, abort, a.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        if (bytes > 0) ptx::mbar_expect_tx(BAR(kCbFullVr + (j & 1)), bytes); else ptx::mbar_arrive(BAR(kCbFullVr + (j & 1)));
      }
      __syncwarp();
      if (box)
        ptx::tma_load_3d(s_base + C::kVr + (j & 1) * C::kKT + 16 * lane * D, &map_v, 0, 0, cur.id * heads + h,
                         BAR(kCbFullVr + (j & 1)));
      last_v = j;
      if (++ks == C::kKStages) ks = 0;
    }
    // no copy is in flight when the CTA exits, however the others ended
    for (int j = max(0, last_k - C::kKStages + 1); j <= last_k; ++j)
      page_drain(BAR(kCbFullK + j % C::kKStages), (j / C::kKStages) & 1, lim);
    for (int j = max(0, last_v - kVStages + 1); j <= last_v; ++j)
      page_drain(BAR(kCbFullVr + (j & 1)), (j >> 1) & 1, lim);
    __syncwarp();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTCols);
  }
}

// Joins the key ranges of split row tiles: one warp per query row and head,
// the ranges in order.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const __grid_constant__ ChunkArgs p) {
  constexpr int C = D / 32;
  ptx::grid_dependency_wait();
  const PagedAttnArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int hq = (int)(w % a.q_heads);
  const long long rb = w / a.q_heads;
  const int i = (int)(rb % a.max_q);
  const long long b = rb / a.max_q;
  if (b >= a.s.batch) return;
  int r0, n;
  seq_rows(a.s, (int)b, r0, n, a.status);
  if (i >= min(n, a.max_q)) return;
  const long long row = (long long)(r0 + i) * a.q_heads + hq, step = (long long)a.s.rows * a.q_heads;
  if (!KVQ_IN_BOUNDS(row, step, a.status, a.bounds_site)) return;
  float top = -CUDART_INF_F;
  for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.part_ml[(s * step + row) * 2]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float base = top > -CUDART_INF_F ? top : 0.f;
  float o[C], l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (s * step + row) * 2);
    // (the sum by two factors: it may stand 75 binades above 2^m)
    const float h = ptx::ex2_approx(0.5f * (ml.x - base)), f = h * h;
    l = fmaf(ml.y * h, h, l);
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(p.part_o[(s * step + row) * D + C * lane + c], f, o[c]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < C; c += 2) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(o[c] * inv, o[c + 1] * inv);
    *reinterpret_cast<uint32_t*>(a.out + row * D + C * lane + c) = *reinterpret_cast<const uint32_t*>(&y);
  }
  if (lane == 0 && a.lse != nullptr) a.lse[row] = lse_of(top, l);
}

}  // namespace
}  // namespace kvq
