// add_norm_launch.h -- internal interface of residual + dropout + norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "philox.h"

namespace ssm66 {
namespace add_norm {

struct Args {
  const void* x;               // (rows, dim) io dtype
  const void* residual;        // nullable, h's type
  const float *weight, *bias;  // nullable (dim)
  void* y;                     // io dtype
  void* h;                     // forwards: nullable; backwards: read
  float *mean, *rstd;          // (rows), nullable forwards; mean unused by the RMS norm
  Drop drop;
  int64_t rows;
  int dim;
  int rms;
  float eps;
  // backwards
  const void *dy, *dh;         // io dtype; h's type, nullable
  void *dx, *dresidual;        // io dtype; h's type, nullable
  float *dweight, *dbias;      // nullable (dim)
  float2* part;                // (blocks, dim)
};
constexpr int64_t kMostDim = 16384;
size_t workspace_bytes(int64_t rows, int64_t dim);  // of the backward with dweight or dbias
hipError_t forward(const Args& p, bool x_f32, bool h_f32, hipStream_t s);
hipError_t backward(const Args& p, bool x_f32, bool h_f32, hipStream_t s);

}  // namespace add_norm
}  // namespace ssm66
