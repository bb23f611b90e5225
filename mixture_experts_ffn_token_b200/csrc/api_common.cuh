// api_common.cuh -- what the files of the C ABI (moe_api.cu,
// operators_api.cu) share: the device check, the configuration check and the
// small helpers of an entry point.
#pragma once

#include <nvtx3/nvToolsExt.h>

#include "kernels.cuh"

namespace moe {

// The current device must be compute capability 10.0 (the library's code is
// sm_100a only) and the driver must expose the tensor-map encoder.
moe_status_t current_device(int* num_sms);

// Host-side checks of a configuration, the same for every entry point.
moe_status_t validate_config(const moe_config_t* c);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(base) + off);
}

// NVTX ranges (MOE_B200_NVTX=1): one per API call and one around the
// enqueue of each kernel, named "moe.<stage>", for a timeline profiler to
// line up with the kernels.  Off by default (no NVTX call is made).
bool nvtx_enabled();

struct NvtxRange {
  const bool on;
  explicit NvtxRange(const char* name) : on(nvtx_enabled()) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxRange() {
    if (on) nvtxRangePop();
  }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace moe
