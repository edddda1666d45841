// gdn_host.h -- host helpers of the layer operators' entry points: argument
// checks and launches.  Every file that includes it has its own copies.
#pragma once
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <initializer_list>
#include <tuple>
#include <type_traits>
#include <utility>

#include "gdn.h"

namespace {

constexpr size_t kWsAlign = 256;
inline size_t align_up(size_t x) { return (x + kWsAlign - 1) & ~(kWsAlign - 1); }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Compute units of the current device (cached per device id; a benign race at
// worst stores the same value twice).
inline int device_cus() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 0;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
  if (dev < 64) cache[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// hipLaunchKernel with the argument tuple converted to the kernel's own types.
template <typename... KArgs, typename... Args>
hipError_t launch(void (*kern)(KArgs...), dim3 grid, dim3 block, hipStream_t s, Args&&... args) {
  std::tuple<KArgs...> t(std::forward<Args>(args)...);
  return std::apply(
      [&](auto&... a) {
        void* argv[] = {(void*)&a...};
        return hipLaunchKernel((const void*)kern, grid, block, argv, 0, s);
      },
      t);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether a grid of that many workgroups can be launched: HIP takes less than 2^32 threads
// per dimension.  Asked for every launch of a call before the first one.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

// Sequence and token counts of a batch: B sequences of T tokens, or (packed) N
// sequences in one row of T tokens.  The rules are gdn_fwd's.
inline gdn_status_t check_batch(int32_t B, int32_t T, int32_t num_seqs, bool packed) {
  if (B < 0 || T < 0) return GDN_ERR_SHAPE;
  if (packed && (B != 1 || num_seqs < 0 || (num_seqs == 0 && T > 0))) return GDN_ERR_SHAPE;
  // token indices are int32, a group of tokens ahead included
  if ((int64_t)B * T > INT32_MAX - 4096) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

}  // namespace
