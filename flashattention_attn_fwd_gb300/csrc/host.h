// Host-side pieces shared by the C ABI entry points (internal header).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "flattn.h"
#include "per_device.h"

namespace fl {

// Everything fl_attn_fwd does after its own set-up: validation, strides,
// kernel parameters, tensor maps and the launch.  `status` is the device
// status word (two uint32) the kernel reports timeouts in, `sm_count` the
// grid cap.  Allocates nothing.
fl_status attn_fwd_launch(const void* q, const void* k, const void* v, void* out, float* lse,
                          const fl_attn_desc* desc, uint32_t* status, int sm_count);

// Argument checks of attn_fwd_launch alone (no CUDA call).
fl_status attn_fwd_check(const void* q, const void* k, const void* v, void* out, float* lse,
                         const fl_attn_desc* desc);

// The current device's SM count and status words, set up on the first call
// per device (FL_ERR_CUDA with a detail on failure).
fl_status device_info(int* sm_count, uint32_t** status);

// FL_OK, or FL_ERR_CUDA with `where` and CUDA's message as the error detail.
fl_status launch_result(const char* where, cudaError_t e);

// The device of the call that this thread is in: below kMaxDevices, set by every
// entry point before it launches (device_info, or the allocation-free call's set-up).
extern thread_local int t_device;

// `step` once on that device (a kernel's attributes and occupancy belong to the
// device): its error until it succeeds there, then cudaSuccess.
template <class Step>
cudaError_t on_this_device(OncePerDevice& once, Step&& step) {
  return once.run(t_device, step);
}

// Launches `kernel` behind the previous kernel of the stream, whose end it waits
// for itself (ptx::wait_prerequisites), so that its set-up runs under that end.
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                           const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fl
