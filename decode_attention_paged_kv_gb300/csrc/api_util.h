// api_util.h -- what the entry points' files share: checks of arguments, the device's
// multiprocessors, the driver's tensor-map encoder.
#pragma once

#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "../../include/dkv.h"

namespace dkv {
namespace api {

constexpr uint64_t kWaitLimitNs = 200000000ull;  // 200 ms per bounded device wait
constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline dkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DKV_OK : DKV_ERR_CUDA; }

inline int out_code(int32_t out_dtype) {
  return out_dtype == DKV_FP32 ? 2 : (out_dtype == DKV_FP16 ? 1 : 0);
}

// Multiprocessor count of the current device (the persistent attention grid).
inline int current_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) cached[dev] = n;
  return n;
}

inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::once_flag g_encode_once;

inline bool get_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// Whether the elements of a tensor that is written -- rows of `inner` elements
// over the dimensions (count, stride) -- all have places of their own.
struct Dim {
  int64_t count, stride;
};
inline bool distinct(int64_t inner, std::initializer_list<Dim> dims) {
  Dim d[3];
  int n = 0;
  for (const Dim& x : dims)
    if (x.count > 1) d[n++] = x;
  std::sort(d, d + n, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t extent = inner;
  for (int i = 0; i < n; ++i) {
    if (d[i].stride < extent) return false;
    extent += (d[i].count - 1) * d[i].stride;
  }
  return true;
}

}  // namespace api
}  // namespace dkv
