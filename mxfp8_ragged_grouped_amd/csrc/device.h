// device.h -- the host's check that the current device is a gfx950, shared by
// the library's entry points.
#ifndef MXW_DEVICE_H
#define MXW_DEVICE_H

#include <hip/hip_runtime.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "mxfp8_wgrad.h"

namespace mxw {

struct DeviceInfo {
  std::atomic<int> state;  // 0: not read yet, 1: gfx950, 2: another device
  int cus;                 // compute units (written before state)
};
inline DeviceInfo g_dev[64];
inline std::mutex g_dev_mutex;  // taken only by the first check of a device

// Reads device properties once per device (no allocation, no stream work);
// after that a check is one atomic load, so calls take no lock.
inline int check_device(int* cus = nullptr) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return MXW_ERR_DEVICE;
  DeviceInfo& d = g_dev[dev];
  int st = d.state.load(std::memory_order_acquire);
  if (st == 0) {
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    st = d.state.load(std::memory_order_relaxed);
    if (st == 0) {
      hipDeviceProp_t prop;
      if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MXW_ERR_DEVICE;
      d.cus = prop.multiProcessorCount;
      st = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
      d.state.store(st, std::memory_order_release);
    }
  }
  if (cus) *cus = d.cus;
  return st == 1 ? MXW_OK : MXW_ERR_DEVICE;
}

}  // namespace mxw

#endif  // MXW_DEVICE_H
