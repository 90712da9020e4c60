// linattn_bf16.hip -- the walks of linear attention over bf16 tensors.
#include "linattn_walk.h"

namespace ssm66 {
namespace linattn {

hipError_t walk_bf16(const WalkArgs& a, Tile t, bool rev, bool dg, bool state, hipStream_t stream) {
  if (t.KP == 64 && t.VB == 32) return launch_walk<1, 64, 32>(a, rev, dg, state, stream);
  if (t.KP == 128 && t.VB == 32) return launch_walk<1, 128, 32>(a, rev, dg, state, stream);
  if (t.KP == 256 && t.VB == 32) return launch_walk<1, 256, 32>(a, rev, dg, state, stream);
  if (t.KP == 64 && t.VB == 64) return launch_walk<1, 64, 64>(a, rev, dg, state, stream);
  if (t.KP == 128 && t.VB == 64) return launch_walk<1, 128, 64>(a, rev, dg, state, stream);
  if (state && t.KP == 64 && t.VB == 128) return launch_walk<1, 64, 128>(a, rev, dg, true, stream);
  if (state && t.KP == 128 && t.VB == 128) return launch_walk<1, 128, 128>(a, rev, dg, true, stream);
  return hipErrorInvalidValue;
}

}  // namespace linattn
}  // namespace ssm66
