// Host-side helpers shared by the entry points.
#pragma once

#include <cuda_runtime.h>

#include "verify_attn.h"

namespace va {

// Remember the CUDA error behind a VA_ERR_CUDA (va_last_cuda_error).
va_status note_cuda(cudaError_t e);

// VA_ERR_INVALID_ARG for a stream of another device than the current one
// (outside stream capture; the default streams are the current device's).
va_status check_stream_device(cudaStream_t s);

}  // namespace va
