// group_norm_launch.h -- internal interface of the group-norm kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm66 {
namespace group_norm {

struct Args {
  const void *x, *z, *dy;        // (batch, rows, C) io dtype; z nullable; dy: backward
  const float *weight, *bias;    // nullable (C)
  float *mean, *rstd;            // (batch, groups): written forwards (nullable), read backwards
  void *y, *dx, *dz;             // io dtype; dz where z is given
  float *dweight, *dbias;        // nullable (C)
  void* ws;
  int64_t batch, rows;
  int C, groups;
  int silu;
  float eps;
  // set by the launch
  int pieces;
  int64_t piece_rows;
};

// whether the grids these sizes need exist
bool fits(const Args& p, bool f32, bool bwd);
// enough for any alignment of the tensors (it sets the width of the accesses
// and with it the launch)
size_t workspace_bytes(const Args& p, bool f32, bool bwd);
hipError_t forward(const Args& p, bool f32, hipStream_t s);
hipError_t backward(const Args& p, bool f32, hipStream_t s);

}  // namespace group_norm
}  // namespace ssm66
