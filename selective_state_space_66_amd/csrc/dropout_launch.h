// dropout_launch.h -- internal interface of dropout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "philox.h"

namespace ssm66 {
namespace dropout {

struct Args {
  const void *x, *residual;  // io type; y's type, nullable
  void* y;
  int64_t n;
  Drop drop;
};
hipError_t run(const Args& p, bool x_f32, bool y_f32, hipStream_t s);

}  // namespace dropout
}  // namespace ssm66
