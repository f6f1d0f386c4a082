// Device helpers of the serving operators.
#pragma once

#include <atomic>

#include "q4_device.cuh"
#include "q4_kv.h"

namespace q4 {

// Device status bit: a NaN or an infinity was given to the cache (Q4_DEVERR_VALUE of the public header).
constexpr unsigned kDevErrValue = 0x4u;

// Lets `kernel` use `bytes` of dynamic shared memory; asked once for each
// device (`done`: a bit for each, one word a kernel).
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Four codes to two pairs of fp16: u = code + 128 as the low byte of 1024 + u, minus 1152, exact.
__device__ __forceinline__ uint32_t sub1152(uint32_t x) {
  uint32_t y;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xE480E480u));
  return y;
}
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = sub1152(__byte_perm(u, 0x64646464u, 0x4140));
  hi = sub1152(__byte_perm(u, 0x64646464u, 0x4342));
}

// The number of j in [1, n] with f(j) <= i, f non-decreasing: the whole warp
// searches 32 probes at a time (one step up to n = 32, two up to 1024).
template <typename F>
__device__ __forceinline__ int warp_count_le(int n, int i, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = (lane + 1) * step;
    const bool ok = at <= n && f(lo + at) <= i;
    const int c = __popc(__ballot_sync(0xffffffffu, ok));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  return lo;
}

// Row of codes (token `pos`, head h) in units of rows of `dim`, or -1 where
// the page table has no valid page for it.
__device__ __forceinline__ long long kv_row(const KvView& c, const int32_t* table,
                                            long long table_stride, int b, int pos, int h) {
  const int pi = pos >> c.page_log2;
  if (pi >= table_stride) return -1;
  const int pg = table[b * table_stride + pi];
  if (pg < 0 || pg >= c.pages) return -1;
  return (static_cast<long long>(pg) * c.heads + h) * c.page + (pos & (c.page - 1));
}

}  // namespace q4
