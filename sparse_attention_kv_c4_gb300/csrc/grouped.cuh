// grouped.cuh -- what the calls of a dense layer of grouped heads share: packed
// sequences (offsets, their search), the 8-bit cache's layout and small conversions.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "fm_common.cuh"
#include "fm_internal.h"

namespace fm {

constexpr int kKvPage = FM_KV_PAGE;
constexpr int kKvBlock = FM_KV_BLOCK;
constexpr int kBlocksPerPage = kKvPage / kKvBlock;
constexpr int kMaxTable = 1 << 19;

FM_DEV float2 bf16x2_floats(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
FM_DEV uint32_t floats_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// mbar_wait in few instructions: these kernels wait in many places, and what leaves the instruction cache
// costs every role (the tensor-core kernel with mbar_wait's unrolled polls was 120 KB of code).
FM_DEV bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
#pragma unroll 1
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if ((n & 31) != 0) continue;
    const bool late = globaltimer() - t0 > FM_WAIT_LIMIT_NS;
    if (late && *abort == 0) atomicOr(status, FM_DEV_TIMEOUT);
    if (late) *abort = 1;
    if (*abort != 0) return false;
  }
  return true;
}

// The same with its loop out of line, for roles that have registers to spare at a call.
static __device__ __noinline__ bool wait_poll(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  return wait_bar(bar, parity, abort, status);
}
FM_DEV bool wait_call(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  return mbar_try_wait(bar, parity) || wait_poll(bar, parity, abort, status);
}

// Offset i of packed sequences, kept within the call's rows whatever it holds.
FM_DEV int offset_at(const int32_t* cu, int i, int rows) { return min(max(cu[i], 0), rows); }

// The largest i of 0 .. n - 1 with key(i) <= x, for a non-decreasing key with key(0) <= x
// (0 where that does not hold), by a whole warp: 32 probes at a time, so that up to
// 1024 sequences take two dependent loads instead of ten.
template <class Key>
FM_DEV int warp_find(int n, int64_t x, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && key(lo + at) <= x;
    int c = __popc(__ballot_sync(0xffffffffu, le));
    c = c > 0 ? c - 1 : 0;
    lo += c * step;
    n = min(step, n - c * step);
  }
  return lo;
}

// The kinds of argument that the three calls have in common; nullptr or what is wrong.
inline const char* bad_heads(int n_h, int n_k, int d) {
  if (n_h < 1 || n_h > 1024 || n_k < 1 || n_h % n_k != 0 || n_h / n_k > 128)
    return "1 <= n_h <= 1024, n_h a multiple of n_k, n_h / n_k <= 128";
  if (d < 16 || d > 128 || d % 16 != 0) return "d: a multiple of 16 up to 128";
  return nullptr;
}
inline bool bad_rows(const void* x, int64_t stride, int heads, int d) {
  return !x || !aligned(x, 16) || stride < (int64_t)heads * d || stride % 8 != 0 || stride > (int64_t(1) << 38);
}
inline const char* bad_cache(const void* k_pool, const void* v_pool, const void* k_scale, const void* v_scale, int64_t P,
                             int64_t page_stride, int64_t scale_stride, const int32_t* table, int B, int R, int n_k, int d) {
  if (P < 0 || P > (int64_t(1) << 25) || B < 0 || B > (1 << 24) || R < 0 || R > kMaxTable)
    return "sizes: 0 <= P <= 2^25, 0 <= B <= 2^24, 0 <= R <= 2^19";
  if (page_stride < (int64_t)n_k * kKvPage * d || page_stride % 16 != 0 || page_stride >= (int64_t(1) << 38))
    return "page_stride: a multiple of 16 bytes, at least n_k * 64 * d";
  if (scale_stride < (int64_t)n_k * kBlocksPerPage || scale_stride % 4 != 0 || scale_stride >= (int64_t(1) << 38))
    return "scale_stride: a multiple of 4, at least 4 n_k";
  if (P > 0 && (!k_pool || !v_pool || !k_scale || !v_scale)) return "a pool or its scales are NULL";
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
    return "pools and scales must be 16-byte aligned";
  if ((B > 0 && R > 0 && !table) || !aligned(table, 4)) return "page_table is NULL or misaligned";
  return nullptr;
}

// Launches a kernel that needs `smem` bytes of shared memory, which has to be said once in a device's context
// (1.3 us a time).  `said` has a bit for each device where it was; a launch that is refused all the same (a
// reset has ended that context) says it again.
template <class... Params, class... Args>
cudaError_t launch_with_smem(std::atomic<uint64_t>& said, int smem, const cudaLaunchConfig_t& cfg, void (*kernel)(Params...),
                             const Args&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  for (bool again = dev < 64 && (said.load() >> dev & 1) != 0;; again = false) {
    if (!again) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      if (dev < 64) said.fetch_or(uint64_t(1) << dev);
    }
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaErrorInvalidValue || !again) return e;
    cudaGetLastError();
  }
}

}  // namespace fm
