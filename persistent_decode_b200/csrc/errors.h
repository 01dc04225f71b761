// What the translation units behind the C ABI share: the thread's error text and
// the checks that every stand-alone operator makes before it enqueues anything.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/xlpk.h"

namespace xlpk {

// The status of a failed CUDA call, its text kept for xlpk_last_cuda_error.
xlpk_status cuda_fail(cudaError_t e, const char* what);
// `st`, with `why` kept for xlpk_last_cuda_error.
xlpk_status refuse(xlpk_status st, const char* why) noexcept;

#define XLPK_CUDA(call)                                       \
  do {                                                        \
    cudaError_t e_ = (call);                                  \
    if (e_ != cudaSuccess) return ::xlpk::cuda_fail(e_, #call); \
  } while (0)

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// SM count of the current device, which must be an sm_100.
xlpk_status current_sms(int* sms);

}  // namespace xlpk
