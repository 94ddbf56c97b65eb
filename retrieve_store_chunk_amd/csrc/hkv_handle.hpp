// The layout handle behind the C ABI, and what its entry points share: the
// thread's error message, the trace switch, the stream's device.  Defined in
// hkv_api.cpp.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "hkv.h"
#include "hkv_plan.hpp"

struct hkv_layout {
  hkv::Plan plan;
  // The plan's constant tables as the kernels read them: layer placements
  // (padded to 256 bytes), then the per-chunk work items.
  std::vector<uint8_t> table_image;
  // Never reused by another layout of the process: names the tables that the
  // static scratch of hkv_move_chunks_noalloc holds.
  uint64_t serial = 0;
  // The constant tables in the memory of each device the layout has been
  // used on, uploaded by the first call there and freed with the layout.
  mutable std::mutex mu;
  mutable std::map<int, void*> dev_tables;
  ~hkv_layout();
};

namespace hkv {

// Remembers `msg` as the calling thread's last error and returns `st`.
hkv_status set_error(hkv_status st, const std::string& msg);
hkv_status hip_error(hipError_t e, const char* what);

// HKV_TRACE=1 in the environment: one line on stderr per layout and per
// call (the layout's N, chunk size and placements; a call's chunks, launches,
// work items and bytes), like the engine's own log line naming the block size
// it settled on.
bool trace_on();

// Makes `dev` current for the scope, restoring the previous device after.
struct DeviceScope {
  int prev = -1;
  hipError_t err = hipSuccess;
  explicit DeviceScope(int dev) {
    err = hipGetDevice(&prev);
    if (err == hipSuccess && prev != dev) err = hipSetDevice(dev);
  }
  ~DeviceScope() {
    int cur = -1;
    if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
  }
};

// The device a call's work goes to: the stream's, or the current one for
// the default stream.
hkv_status stream_device(hipStream_t stream, int* dev);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace hkv
