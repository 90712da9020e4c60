// lm_api.hip -- the C ABI declared in include/ssm66_lm.h: argument validation
// before any HIP call, then the launches.
#include <stdint.h>

#include <initializer_list>

#include "../../include/ssm66_lm.h"
#include "grad_clip_launch.h"
#include "group_norm_launch.h"
#include "linattn_launch.h"

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// the product of non-negative factors within INT64_MAX / 8 (so byte counts
// stay in range too)
bool product(int64_t* out, std::initializer_list<int64_t> f) {
  __int128 r = 1;
  for (int64_t x : f) {
    r *= x;
    if (r > INT64_MAX / 8) return false;
  }
  *out = (int64_t)r;
  return true;
}

int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

int linattn_shape(int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                  int64_t dv, int io_dtype) {
  if (batch < 0 || seqlen < 0 || nheads < 0 || kheads < 1 || dk < 1 || dv < 1) return SSM_ERR_SHAPE;
  if (nheads % kheads != 0) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  int64_t t;
  if (!product(&t, {batch, seqlen, nheads, dk}) || !product(&t, {batch, seqlen, nheads, dv}) ||
      !product(&t, {batch, nheads, dk, dv, 64}))
    return SSM_ERR_SHAPE;
  return SSM_OK;
}

int linattn_limits(int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                   int64_t dv, bool backward) {
  // 16-byte pieces of a row, the widest tile of the kernels, 32-bit offsets
  // within a chunk, 32-bit block numbers (at most 64 spans and 16 slices)
  if (dk % 8 != 0 || dv % 8 != 0 || dk > 256 || dv > 256) return SSM_ERR_UNSUPPORTED;
  const int64_t widest = (int64_t)1 << 22;
  if (nheads > widest || nheads * dv > widest || kheads * dk > widest) return SSM_ERR_UNSUPPORTED;
  // gradients of shared keys have a row per head before they are added
  if (backward && nheads * dk > widest) return SSM_ERR_UNSUPPORTED;
  if (batch > 0x7fffffff || batch * nheads > 0x7fffffff / 1024) return SSM_ERR_UNSUPPORTED;
  if (seqlen > (int64_t)64 * 0x7fffff) return SSM_ERR_UNSUPPORTED;
  // the sums over shared heads: one thread for four columns
  if (batch * kheads > 0 && seqlen > (int64_t)0x7fffffff * 256 / (batch * kheads * (dk / 4)))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm66::linattn::Problem problem(const void* q, const void* k, const void* v, const float* log_decay,
                                float scale, const float* h0, const int32_t* seq_lens,
                                const uint8_t* reset, int64_t batch, int64_t seqlen,
                                int64_t nheads, int64_t kheads, int64_t dk, int64_t dv,
                                int io_dtype) {
  ssm66::linattn::Problem p;
  p.q = q; p.k = k; p.v = v; p.log_decay = log_decay; p.h0 = h0; p.seq_lens = seq_lens;
  p.reset = reset; p.batch = batch; p.L = seqlen; p.H = (int)nheads; p.Hk = (int)kheads;
  p.Dk = (int)dk; p.Dv = (int)dv; p.scale = scale; p.f32 = io_dtype == SSM_F32;
  return p;
}

int norm_shape(int64_t batch, int64_t rows, int64_t channels, int64_t groups, int io_dtype) {
  if (batch < 0 || rows < 0 || channels < 1 || groups < 1 || channels % groups != 0) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  int64_t t;
  if (!product(&t, {batch, rows, channels}) || !product(&t, {batch, channels})) return SSM_ERR_SHAPE;
  if (channels > ((int64_t)1 << 22)) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

ssm66::group_norm::Args norm_args(int64_t batch, int64_t rows, int64_t channels, int64_t groups) {
  ssm66::group_norm::Args a = {};
  a.batch = batch; a.rows = rows; a.C = (int)channels; a.groups = (int)groups;
  return a;
}

}  // namespace

extern "C" {

size_t ssm_group_norm_workspace_size(int64_t batch, int64_t rows, int64_t channels,
                                     int64_t groups, int backward, int io_dtype) {
  if (norm_shape(batch, rows, channels, groups, io_dtype) != SSM_OK) return 0;
  ssm66::group_norm::Args a = norm_args(batch, rows, channels, groups);
  if (!ssm66::group_norm::fits(a, io_dtype == SSM_F32, backward != 0)) return 0;
  return ssm66::group_norm::workspace_bytes(a, io_dtype == SSM_F32, backward != 0);
}

int ssm_group_norm_fwd(const void* x, const float* weight, const float* bias, const void* z,
                       int act, float eps, void* y, float* mean, float* rstd, void* workspace,
                       size_t workspace_bytes, int64_t batch, int64_t rows, int64_t channels,
                       int64_t groups, int io_dtype, void* stream) {
  const int st = norm_shape(batch, rows, channels, groups, io_dtype);
  if (st != SSM_OK) return st;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return SSM_ERR_FLAG;
  if (batch == 0 || rows == 0) return SSM_OK;
  if (!x || !y) return SSM_ERR_NULL;
  const size_t es = io_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(z, es)) return SSM_ERR_ALIGN;
  const void* p4[4] = {weight, bias, mean, rstd};
  for (const void* q : p4)
    if (!aligned(q, 4)) return SSM_ERR_ALIGN;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm66::group_norm::Args a = norm_args(batch, rows, channels, groups);
  const bool f32 = io_dtype == SSM_F32;
  if (!ssm66::group_norm::fits(a, f32, false)) return SSM_ERR_UNSUPPORTED;
  const size_t need = ssm66::group_norm::workspace_bytes(a, f32, false);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  a.x = x; a.z = z; a.y = y; a.weight = weight; a.bias = bias; a.mean = mean; a.rstd = rstd;
  a.silu = act == SSM_ACT_SILU; a.eps = eps; a.ws = workspace;
  return status(ssm66::group_norm::forward(a, f32, (hipStream_t)stream));
}

int ssm_group_norm_bwd(const void* x, const float* weight, const float* bias, const void* z,
                       int act, const float* mean, const float* rstd, const void* dy, void* dx,
                       float* dweight, float* dbias, void* dz, void* workspace,
                       size_t workspace_bytes, int64_t batch, int64_t rows, int64_t channels,
                       int64_t groups, int io_dtype, void* stream) {
  const int st = norm_shape(batch, rows, channels, groups, io_dtype);
  if (st != SSM_OK) return st;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return SSM_ERR_FLAG;
  if (batch > 0 && rows > 0 && (!x || !dy || !dx || !mean || !rstd || (z && !dz))) return SSM_ERR_NULL;
  const size_t es = io_dtype == SSM_BF16 ? 2 : 4;
  const void* io[5] = {x, z, dy, dx, dz};
  for (const void* q : io)
    if (!aligned(q, es)) return SSM_ERR_ALIGN;
  const void* p4[6] = {weight, bias, mean, rstd, dweight, dbias};
  for (const void* q : p4)
    if (!aligned(q, 4)) return SSM_ERR_ALIGN;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  ssm66::group_norm::Args a = norm_args(batch, rows, channels, groups);
  const bool f32 = io_dtype == SSM_F32;
  if (!ssm66::group_norm::fits(a, f32, true)) return SSM_ERR_UNSUPPORTED;
  const size_t need = ssm66::group_norm::workspace_bytes(a, f32, true);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  a.x = x; a.z = z; a.dy = dy; a.dx = dx; a.dz = dz; a.weight = weight; a.bias = bias;
  a.mean = (float*)mean; a.rstd = (float*)rstd; a.dweight = dweight; a.dbias = dbias;
  a.silu = act == SSM_ACT_SILU; a.ws = workspace;
  return status(ssm66::group_norm::backward(a, f32, (hipStream_t)stream));
}

size_t ssm_clip_grad_norm_workspace_size(int64_t ntensors) {
  if (ntensors < 0 || ntensors > ((int64_t)1 << 24)) return 0;
  return ssm66::grad_clip::workspace_bytes(ntensors);
}

int ssm_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* counts,
                       const int32_t* io_dtypes, int64_t ntensors, float max_norm, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (ntensors < 0) return SSM_ERR_SHAPE;
  if (ntensors > ((int64_t)1 << 24)) return SSM_ERR_UNSUPPORTED;
  if (!(max_norm >= 0.0f)) return SSM_ERR_FLAG;
  if (!norm || (ntensors > 0 && (!grads || !outs || !counts || !io_dtypes))) return SSM_ERR_NULL;
  for (int64_t i = 0; i < ntensors; ++i) {
    if (counts[i] < 0) return SSM_ERR_SHAPE;
    if (counts[i] > ((int64_t)1 << 38)) return SSM_ERR_UNSUPPORTED;  // chunk numbers are 32-bit
    if (io_dtypes[i] != SSM_F32 && io_dtypes[i] != SSM_BF16) return SSM_ERR_DTYPE;
    if (counts[i] == 0) continue;
    if (!grads[i] || !outs[i]) return SSM_ERR_NULL;
    const size_t es = io_dtypes[i] == SSM_BF16 ? 2 : 4;
    if (!aligned(grads[i], es) || !aligned(outs[i], es)) return SSM_ERR_ALIGN;
  }
  if (!aligned(norm, 4) || !aligned(workspace, 256)) return SSM_ERR_ALIGN;
  const size_t need = ssm66::grad_clip::workspace_bytes(ntensors);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  ssm66::grad_clip::Call c;
  c.grads = grads; c.outs = outs; c.counts = counts; c.io_dtypes = io_dtypes; c.n = ntensors;
  c.max_norm = max_norm; c.norm = norm; c.ws = workspace;
  return status(ssm66::grad_clip::run(c, (hipStream_t)stream));
}


size_t ssm_linattn_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads,
                                      int64_t kheads, int64_t dk, int64_t dv, int io_dtype) {
  if (linattn_shape(batch, seqlen, nheads, kheads, dk, dv, io_dtype) != SSM_OK ||
      linattn_limits(batch, seqlen, nheads, kheads, dk, dv, false) != SSM_OK)
    return 0;
  return ssm66::linattn::fwd_workspace(problem(nullptr, nullptr, nullptr, nullptr, 1.0f, nullptr,
                                               nullptr, nullptr, batch, seqlen, nheads, kheads, dk,
                                               dv, io_dtype));
}

size_t ssm_linattn_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t nheads,
                                      int64_t kheads, int64_t dk, int64_t dv,
                                      int need_dlog_decay, int io_dtype) {
  if (linattn_shape(batch, seqlen, nheads, kheads, dk, dv, io_dtype) != SSM_OK ||
      linattn_limits(batch, seqlen, nheads, kheads, dk, dv, true) != SSM_OK)
    return 0;
  return ssm66::linattn::bwd_workspace(problem(nullptr, nullptr, nullptr, nullptr, 1.0f, nullptr,
                                               nullptr, nullptr, batch, seqlen, nheads, kheads, dk,
                                               dv, io_dtype),
                                       need_dlog_decay != 0);
}

int ssm_linattn_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const float* h0, const int32_t* seq_lens, const uint8_t* reset,
                    void* o, float* last_state, void* workspace, size_t workspace_bytes,
                    int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                    int64_t dv, int io_dtype, void* stream) {
  int st = linattn_shape(batch, seqlen, nheads, kheads, dk, dv, io_dtype);
  if (st != SSM_OK) return st;
  if (batch == 0 || nheads == 0) return SSM_OK;
  if (!log_decay || (seqlen > 0 && (!q || !k || !v || !o))) return SSM_ERR_NULL;
  if ((st = linattn_limits(batch, seqlen, nheads, kheads, dk, dv, false)) != SSM_OK) return st;
  const void* p16[6] = {q, k, v, o, h0, last_state};
  for (const void* x : p16)
    if (!aligned(x, 16)) return SSM_ERR_ALIGN;
  if (!aligned(log_decay, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256)) return SSM_ERR_ALIGN;
  if (h0 && h0 == last_state) return SSM_ERR_FLAG;  // every slice of a head reads h0 on its own
  const ssm66::linattn::Problem p = problem(q, k, v, log_decay, scale, h0, seq_lens, reset, batch,
                                            seqlen, nheads, kheads, dk, dv, io_dtype);
  const size_t need = ssm66::linattn::fwd_workspace(p);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  return status(ssm66::linattn::forward(p, {o, last_state}, workspace, (hipStream_t)stream));
}

int ssm_linattn_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                    float scale, const float* h0, const int32_t* seq_lens, const uint8_t* reset,
                    const void* do_, const float* dlast, void* dq, void* dk_, void* dv_,
                    float* dlog_decay, float* dh0, void* workspace, size_t workspace_bytes,
                    int64_t batch, int64_t seqlen, int64_t nheads, int64_t kheads, int64_t dk,
                    int64_t dv, int io_dtype, void* stream) {
  int st = linattn_shape(batch, seqlen, nheads, kheads, dk, dv, io_dtype);
  if (st != SSM_OK) return st;
  if (nheads == 0) return SSM_OK;
  if (batch > 0 && !log_decay) return SSM_ERR_NULL;
  if (batch > 0 && seqlen > 0 && (!q || !k || !v || !do_ || !dq || !dk_ || !dv_)) return SSM_ERR_NULL;
  if ((st = linattn_limits(batch, seqlen, nheads, kheads, dk, dv, true)) != SSM_OK) return st;
  const void* p16[10] = {q, k, v, do_, dq, dk_, dv_, h0, dlast, dh0};
  for (const void* x : p16)
    if (!aligned(x, 16)) return SSM_ERR_ALIGN;
  const void* p4[3] = {log_decay, seq_lens, dlog_decay};
  for (const void* x : p4)
    if (!aligned(x, 4)) return SSM_ERR_ALIGN;
  if (!aligned(workspace, 256)) return SSM_ERR_ALIGN;
  if (dh0 && (dh0 == dlast || dh0 == h0)) return SSM_ERR_FLAG;  // each is read on its own
  const ssm66::linattn::Problem p = problem(q, k, v, log_decay, scale, h0, seq_lens, reset, batch,
                                            seqlen, nheads, kheads, dk, dv, io_dtype);
  const size_t need = ssm66::linattn::bwd_workspace(p, dlog_decay != nullptr);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  return status(ssm66::linattn::backward(p, {do_, dlast, dq, dk_, dv_, dlog_decay, dh0}, workspace,
                                         (hipStream_t)stream));
}

int ssm_linattn_step(float* state, const void* q, const void* k, const void* v,
                     const float* log_decay, float scale, void* o, int64_t batch,
                     int64_t nheads, int64_t kheads, int64_t dk, int64_t dv, int io_dtype,
                     void* stream) {
  const int st = linattn_shape(batch, 1, nheads, kheads, dk, dv, io_dtype);
  if (st != SSM_OK) return st;
  if (batch == 0 || nheads == 0) return SSM_OK;
  if (!state || !q || !k || !v || !log_decay || !o) return SSM_ERR_NULL;
  if (dk % 8 != 0 || dk > 256) return SSM_ERR_UNSUPPORTED;
  const int64_t most = 0x7fffffff;
  if (dv > 1 << 30) return SSM_ERR_UNSUPPORTED;  // rows of a block past the last one stay 32-bit
  if (nheads > most || batch * nheads > most / ((dv + 3) / 4)) return SSM_ERR_UNSUPPORTED;
  const size_t es = io_dtype == SSM_BF16 ? 2 : 4;
  if (!aligned(state, 16) || !aligned(q, 16) || !aligned(k, 16)) return SSM_ERR_ALIGN;
  if (!aligned(v, es) || !aligned(o, es) || !aligned(log_decay, 4)) return SSM_ERR_ALIGN;
  ssm66::linattn::StepArgs a;
  a.state = state; a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.o = o;
  a.batch = batch; a.H = (int)nheads; a.Hk = (int)kheads; a.Dk = (int)dk; a.Dv = (int)dv;
  a.scale = scale; a.f32 = io_dtype == SSM_F32;
  return status(ssm66::linattn::step(a, (hipStream_t)stream));
}

}  // extern "C"
