// layer_api.hip -- the C ABI declared in include/ssm66_layer.h: argument
// validation before any HIP call, then the launches.
#include <stdint.h>

#include <initializer_list>

#include "../../include/ssm66_layer.h"
#include "gated_scan_launch.h"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool aligned_all(size_t a, std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned(p, a)) return false;
  return true;
}

// whether the product of non-negative factors is within INT64_MAX / 8 (so byte
// counts stay in range too)
bool product_fits(std::initializer_list<int64_t> f) {
  __int128 r = 1;
  for (int64_t x : f) {
    r *= x;
    if (r > INT64_MAX / 8) return false;
  }
  return true;
}

int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

size_t width(int io_dtype) { return io_dtype == SSM_BF16 ? 2 : 4; }

int scan_shape(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (batch < 0 || seqlen < 0 || dim < 0) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  return product_fits({batch, seqlen, dim}) && product_fits({batch, dim}) ? SSM_OK : SSM_ERR_SHAPE;
}

ssm66::gated_scan::Args scan_args(const void* x, const void* r, const void* i, const float* decay,
                                  const int32_t* seq_lens, const uint8_t* reset, int64_t batch,
                                  int64_t seqlen, int64_t dim, void* ws) {
  ssm66::gated_scan::Args a = {};
  a.x = x; a.r = r; a.i = i; a.decay = decay; a.seq_lens = seq_lens; a.reset = reset;
  a.batch = batch; a.L = seqlen; a.dim = (int)dim; a.ws = ws;
  return a;
}

}  // namespace

extern "C" {

size_t ssm_gated_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int backward,
                                     int need_ddecay) {
  if (scan_shape(batch, seqlen, dim, SSM_F32) != SSM_OK || batch == 0 || dim == 0) return 0;
  if (!ssm66::gated_scan::fits(batch, seqlen, dim)) return 0;
  return ssm66::gated_scan::workspace_bytes(batch, seqlen, dim, backward != 0, need_ddecay != 0);
}

int ssm_gated_scan_fwd(const void* x, const void* r, const void* i, const float* decay,
                       const float* h0, const int32_t* seq_lens, const uint8_t* reset, void* y,
                       float* last_state, float* states, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, void* stream) {
  const int st = scan_shape(batch, seqlen, dim, io_dtype);
  if (st != SSM_OK) return st;
  if (batch == 0 || dim == 0) return SSM_OK;
  if (!decay || (seqlen > 0 && (!x || !r || !i || !y))) return SSM_ERR_NULL;
  if (!ssm66::gated_scan::fits(batch, seqlen, dim)) return SSM_ERR_UNSUPPORTED;
  if (!aligned_all(width(io_dtype), {x, r, i, y})) return SSM_ERR_ALIGN;
  if (!aligned_all(4, {decay, h0, seq_lens, last_state, states}) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (h0 && h0 == last_state) return SSM_ERR_FLAG;  // several blocks read h0 on their own
  const size_t need = ssm66::gated_scan::workspace_bytes(batch, seqlen, dim, false, false);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  ssm66::gated_scan::Args a = scan_args(x, r, i, decay, seq_lens, reset, batch, seqlen, dim, workspace);
  a.h0 = h0; a.y = y; a.last_state = last_state; a.states = seqlen > 0 ? states : nullptr;
  return status(ssm66::gated_scan::forward(a, io_dtype == SSM_F32, (hipStream_t)stream));
}

int ssm_gated_scan_bwd(const void* x, const void* r, const void* i, const float* decay,
                       const float* states, const int32_t* seq_lens, const uint8_t* reset,
                       const void* dy, const float* dlast, void* dx, void* dr, void* di,
                       float* ddecay, float* dh0, void* workspace, size_t workspace_bytes,
                       int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, void* stream) {
  const int st = scan_shape(batch, seqlen, dim, io_dtype);
  if (st != SSM_OK) return st;
  if (dim == 0) return SSM_OK;
  if (!decay) return SSM_ERR_NULL;
  if (batch > 0 && seqlen > 0 && (!x || !r || !i || !states || !dy || !dx || !dr || !di)) return SSM_ERR_NULL;
  if (!ssm66::gated_scan::fits(batch, seqlen, dim)) return SSM_ERR_UNSUPPORTED;
  if (!aligned_all(width(io_dtype), {x, r, i, dy, dx, dr, di})) return SSM_ERR_ALIGN;
  if (!aligned_all(4, {decay, states, seq_lens, dlast, ddecay, dh0}) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  if (dh0 && dh0 == dlast) return SSM_ERR_FLAG;  // several blocks read dlast on their own
  const size_t need = batch == 0 ? 0
      : ssm66::gated_scan::workspace_bytes(batch, seqlen, dim, true, ddecay != nullptr);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  ssm66::gated_scan::Args a = scan_args(x, r, i, decay, seq_lens, reset, batch, seqlen, dim, workspace);
  a.states = seqlen > 0 ? (float*)states : nullptr;
  a.dy = dy; a.dlast = dlast; a.dx = dx; a.dr = dr; a.di = di; a.ddecay = ddecay; a.dh0 = dh0;
  return status(ssm66::gated_scan::backward(a, io_dtype == SSM_F32, (hipStream_t)stream));
}

int ssm_gated_scan_step(float* state, const void* x, const void* r, const void* i,
                        const float* decay, void* y, int64_t batch, int64_t dim, int io_dtype,
                        void* stream) {
  const int st = scan_shape(batch, 1, dim, io_dtype);
  if (st != SSM_OK) return st;
  if (batch == 0 || dim == 0) return SSM_OK;
  if (!state || !x || !r || !i || !decay || !y) return SSM_ERR_NULL;
  if (dim > (1 << 24)) return SSM_ERR_UNSUPPORTED;
  if (!aligned_all(width(io_dtype), {x, r, i, y}) || !aligned_all(4, {state, decay})) return SSM_ERR_ALIGN;
  ssm66::gated_scan::StepArgs a;
  a.state = state; a.x = x; a.r = r; a.i = i; a.decay = decay; a.y = y; a.batch = batch; a.dim = (int)dim;
  return status(ssm66::gated_scan::step(a, io_dtype == SSM_F32, (hipStream_t)stream));
}

}  // extern "C"
