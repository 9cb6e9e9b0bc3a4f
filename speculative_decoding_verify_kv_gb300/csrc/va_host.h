// Host-side helpers shared by the entry points.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "verify_attn.h"

namespace va {

// Remember the CUDA error behind a VA_ERR_CUDA (va_last_cuda_error).
va_status note_cuda(cudaError_t e);

// VA_ERR_INVALID_ARG for a stream of another device than the current one
// (outside stream capture; the default streams are the current device's).
va_status check_stream_device(cudaStream_t s);

// Set a kernel's dynamic shared memory limit, once per device (ready: a bit
// for each, a static of the caller).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace va
