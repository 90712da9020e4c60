// linattn_f32.hip -- the walks of linear attention over fp32 tensors.
#include "linattn_walk.h"

namespace ssm66 {
namespace linattn {

hipError_t walk_f32(const WalkArgs& a, Tile t, bool rev, bool dg, bool state, hipStream_t stream) {
  if (t.KP == 64 && t.VB == 32) return launch_walk<3, 64, 32>(a, rev, dg, state, stream);
  if (t.KP == 96 && t.VB == 32) return launch_walk<3, 96, 32>(a, rev, dg, state, stream);
  if (t.KP == 128 && t.VB == 32) return launch_walk<3, 128, 32>(a, rev, dg, state, stream);
  if (t.KP == 256 && t.VB == 16) return launch_walk<3, 256, 16>(a, rev, dg, state, stream);
  return hipErrorInvalidValue;
}

}  // namespace linattn
}  // namespace ssm66
