// Host helpers shared by the library's translation units (defined in api.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "../../include/moe_decode.h"

namespace moe_host {

// Records the CUDA error for moe_last_cuda_error and returns MOE_ERR_CUDA.
int fail(int cuda_error);
// MOE_OK when the current device is compute capability 10.0 (cached per device).
int supported_device();
// Multiprocessors of the current device (cached); 0 when it cannot be asked.
int sms();

// Settings of moe_debug_barrier_test: arrivals that device-side waits expect beyond those that come, and
// the cycles after which they give up.
void test_waits(int* extra_arrivals, long long* limit);

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool float_format(int f) { return f == MOE_FMT_F32 || f == MOE_FMT_BF16; }
inline size_t float_bytes(int f) { return f == MOE_FMT_F32 ? 4 : 2; }

// NVTX range around a library call.
struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

}  // namespace moe_host
