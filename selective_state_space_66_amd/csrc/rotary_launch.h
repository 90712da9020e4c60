// rotary_launch.h -- internal interface of the rotary positions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm66 {
namespace rotary {

struct Args {
  const void *q, *k;         // (batch, L, H | Hk, D) io dtype; k nullable with Hk = 0
  void *qo, *ko;             // like q, k, and may be them
  const float* freqs;        // (pairs)
  const int32_t* positions;  // nullable (batch, L): the token's number in its row
  int64_t tokens, L;
  int H, Hk, D, pairs;
  float mscale, sign;        // sign: -1 rotates back
  int interleaved;
  // set by the launch
  int lanes, splits;         // threads of a token along a head, along the heads
};
// whether the grid these sizes need exists
bool fits(int64_t tokens, int heads, int D);
hipError_t run(const Args& p, bool f32, hipStream_t s);

}  // namespace rotary
}  // namespace ssm66
