// grad_clip_launch.h -- internal interface of the gradient-clipping kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm66 {
namespace grad_clip {

struct Call {
  const void* const* grads;  // host arrays of `n` entries
  void* const* outs;
  const int64_t* counts;
  const int32_t* io_dtypes;  // 0: float, 1: bf16
  int64_t n;
  float max_norm;
  float* norm;               // device
  void* ws;                  // device
};

size_t workspace_bytes(int64_t n);
hipError_t run(const Call& c, hipStream_t s);

}  // namespace grad_clip
}  // namespace ssm66
