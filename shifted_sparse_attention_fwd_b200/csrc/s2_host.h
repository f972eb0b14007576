// Host-side state shared by the translation units of the C ABI: the error text, the per-device
// set-up and the tensor-map encoder (defined in s2attn_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "../../include/s2attn.h"

namespace s2host {

constexpr int kMaxDevices = 64;

// Records the text for s2attn_last_error and returns S2ATTN_ERR_CUDA.
s2attn_status cuda_fail(cudaError_t e, const char* what);
// Records a text for s2attn_last_error and returns `status`.
s2attn_status fail(s2attn_status status, const char* text);
// Device address of the current device's error word, its SM count and its ordinal.
s2attn_status device_state(unsigned int** err_word, int* num_sms = nullptr, int* device = nullptr);
// cuTensorMapEncodeTiled, or null with the error text set.
PFN_cuTensorMapEncodeTiled_v12000 encoder();
unsigned long long wait_timeout_ns();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace s2host
