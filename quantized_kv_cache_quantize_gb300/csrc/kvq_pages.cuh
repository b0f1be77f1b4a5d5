// Device helpers of the paged 8-bit cache: its scale rule, its codes, and
// reading tables, lengths and offsets without trusting them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kvq_pages.h"
#include "kvq_sm100.cuh"

namespace kvq {
namespace {

// Launch that may start while the stream's previous kernel finishes (the
// kernel waits for it before its first global access).
template <typename... Args>
cudaError_t launch_clusters(void (*kern)(Args...), unsigned grid, unsigned cluster, int threads, int smem,
                            cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), unsigned grid, int threads, int smem,
                             cudaStream_t stream, Args... args) {
  return launch_clusters<Args...>(kern, grid, 1u, threads, smem, stream, args...);
}

// Bounded wait on an mbarrier phase: false when the limit ran out (recorded)
// or `abort` (may be null) was raised by another role.
__device__ __noinline__ bool page_wait_slow(uint32_t bar, uint32_t parity, unsigned long long limit_ns,
                                            volatile int* abort, int* status) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 20000u)) {
    if (abort != nullptr && *abort) return false;
    if (ptx::globaltimer() - t0 > limit_ns) {
      if (abort != nullptr) *abort = 1;
      atomicCAS(status, 0, (int)KVQ_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool page_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns,
                                          volatile int* abort, int* status) {
  return ptx::mbar_try_wait(bar, parity) || page_wait_slow(bar, parity, limit_ns, abort, status);
}
// A wait for copies or MMAs this thread has in flight, before it exits:
// bounded, and at least 100 ms long whatever the limit.
__device__ __noinline__ void page_drain(uint32_t bar, uint32_t parity, unsigned long long limit_ns) {
  if (limit_ns < 100000000ull) limit_ns = 100000000ull;
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer() - t0 > limit_ns) return;
  }
}

// 2^e as fp32, -126 <= e <= 127
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// exponent of a stored scale (BF16 bits of a power of two); anything else a
// foreign writer left there is read as some exponent in the range
__device__ __forceinline__ int scale_exp(uint16_t bits) {
  const int e = (int)((bits >> 7) & 255u) - 127;
  return min(max(e, kPageExpMin), kPageExpMax);
}
__device__ __forceinline__ uint16_t scale_bits(int e) { return (uint16_t)((e + 127) << 7); }

// Smallest e with m <= 448 * 2^e (448 = 0.875 * 2^9): m = f * 2^k with f in
// [1, 2) gives e = k - 8, one more when f > 1.75.  m is not negative.
__device__ __forceinline__ int exp_for_max(float m) {
  const uint32_t u = __float_as_uint(m);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kPageExpMin), kPageExpMax);   // zero and fp32 subnormals: the lowest
}
// largest magnitude whose codes do not saturate
__device__ __forceinline__ bool in_code_range(float m) { return m <= 448.f * 1152921504606846976.f; }

// four fp32 values as E4M3 codes (to nearest, ties to even, saturating)
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// two codes as packed FP16 (exact)
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

__device__ __forceinline__ void page_error(int* status) {
  atomicCAS(status, 0, (int)KVQ_ERR_PAGE);
}

// rows [r0, r0 + n) of sequence b, cut to the packed tensor
__device__ __forceinline__ void seq_rows(const PageSeqs& s, int b, int& r0, int& n, int* status) {
  if (s.offsets == nullptr) {
    r0 = b;
    n = 1;
    return;
  }
  const int o0 = __ldg(s.offsets + b), o1 = __ldg(s.offsets + b + 1);
  r0 = min(max(o0, 0), s.rows);
  n = max(min(max(o1, 0), s.rows) - r0, 0);
  if (o0 < 0 || o1 < o0 || o1 > s.rows) page_error(status);
}

__device__ __forceinline__ int seq_len(const PageSeqs& s, int b, int shift, int* status) {
  const int len = __ldg(s.lens + b);
  const long long most = (long long)s.width << shift;
  if (len < 0 || len > most) page_error(status);
  return (int)min((long long)max(len, 0), most);
}

// page of entry p of sequence b, or -1 (recorded) when it is none of the pool's
__device__ __forceinline__ int seq_page(const PageSeqs& s, int b, int p, int n_pages, int* status) {
  const int id = __ldg(s.table + (long long)b * s.stride + p);
  if ((unsigned)id < (unsigned)n_pages) return id;
  page_error(status);
  return -1;
}

}  // namespace
}  // namespace kvq
