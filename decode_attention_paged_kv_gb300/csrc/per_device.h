// per_device.h -- a number that is found out once a device.
#pragma once

#include <atomic>

namespace dkv {

constexpr int kMaxDevices = 64;  // devices whose numbers are kept
using PerDevice = std::atomic<int>[kMaxDevices];  // 0: not known yet

// The number of device `dev`, by compute(int*) -> status on the first call for it;
// a failure is returned and not kept.  compute also does what has to be done once a
// device (an attribute of a kernel belongs to the device that was current when it
// was set).  Threads that meet here compute the same number.
template <typename Status, typename F>
Status per_device(PerDevice& known, int dev, Status ok, int* out, const F& compute) {
  const bool kept = dev >= 0 && dev < kMaxDevices;
  if (kept) {
    const int n = known[dev].load(std::memory_order_acquire);
    if (n > 0) {
      *out = n;
      return ok;
    }
  }
  int n = 0;
  const Status st = compute(&n);
  if (st != ok) return st;
  if (kept) known[dev].store(n, std::memory_order_release);
  *out = n;
  return ok;
}

}  // namespace dkv
