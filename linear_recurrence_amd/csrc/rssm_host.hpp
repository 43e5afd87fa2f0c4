// Host-side helpers shared by the C-ABI entry points.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "replayssm.h"

namespace rssm {

// Dynamic LDS a decode workgroup may request.
constexpr size_t kMaxLds = 64 * 1024;

static inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

static inline bool valid_dtype(int32_t t) { return t == RSSM_F32 || t == RSSM_BF16; }

// A launch holds fewer than 2^32 threads.
static inline bool grid_fits(long grid, long threads) { return grid * threads < (1L << 32); }

// Whether any of so many rows of len bytes, step bytes apart, shares memory with the
// bytes of out.
static inline bool rows_meet(const void* in, long step, long len, long rows, const void* out, long bytes) {
  if (!in || !out || rows == 0) return false;
  const intptr_t a = reinterpret_cast<intptr_t>(in), b = reinterpret_cast<intptr_t>(out);
  // the first row that ends behind the output's start
  const long k = a + len > b ? 0 : (b - a - len) / step + 1;
  return k < rows && a + k * step < b + bytes;
}

// Launch with the error code of the launch itself (not a stale one left in
// the thread's last-error slot by earlier runtime calls).
template <typename Args>
static inline int launch_kernel(const void* fn, unsigned grid, unsigned block,
                                size_t lds, hipStream_t stream, const Args& a) {
  void* kargs[] = {const_cast<Args*>(&a)};
  const hipError_t e = hipLaunchKernel(fn, dim3(grid), dim3(block), kargs, lds, stream);
  return e == hipSuccess ? RSSM_OK : RSSM_ELAUNCH;
}

}  // namespace rssm
