// layer_api.hip -- the C ABI declared in include/ssm66_layer.h: argument
// validation before any HIP call, then the launches.
#include <stdint.h>

#include <initializer_list>

#include "../../include/ssm66_layer.h"
#include "add_norm_launch.h"
#include "dropout_launch.h"
#include "gated_scan_launch.h"
#include "rotary_launch.h"

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

// A tensor's memory; NULL has none.
struct Span { const void* p; size_t bytes; };
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
// whether no output shares memory with an input or with another output
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* q = outs.begin(); q != o; ++q)
      if (meet(*o, *q)) return false;
    for (const Span& i : ins)
      if (meet(*o, i)) return false;
  }
  return true;
}

// whether an output shares no memory with an input, or lies in its place value by value
bool apart_or_over(const Span& out, const Span& in) {
  return !meet(out, in) || (out.p == in.p && out.bytes == in.bytes);
}

int status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

size_t width(int io_dtype) { return io_dtype == SSM_BF16 ? 2 : 4; }

int scan_shape(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (batch < 0 || seqlen < 0 || dim < 0) return SSM_ERR_SHAPE;
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_DTYPE;
  return product_fits({batch, seqlen, dim}) && product_fits({batch, dim}) ? SSM_OK : SSM_ERR_SHAPE;
}

size_t kept_states(int64_t seqlen) {
  return (size_t)(seqlen / ssm66::gated_scan::kKeep + (seqlen % ssm66::gated_scan::kKeep != 0));
}

ssm66::gated_scan::Args scan_args(const void* x, const void* r, const void* i, const float* decay,
                                  const int32_t* seq_lens, const uint8_t* reset, int64_t batch,
                                  int64_t seqlen, int64_t dim, void* ws) {
  ssm66::gated_scan::Args a = {};
  a.x = x; a.r = r; a.i = i; a.decay = decay; a.seq_lens = seq_lens; a.reset = reset;
  a.batch = batch; a.L = seqlen; a.dim = (int)dim; a.ws = ws;
  return a;
}

bool io_type(int t) { return t == SSM_F32 || t == SSM_BF16; }

// sizes, types, rate and norm of the add_norm calls
int norm_args(int64_t rows, int64_t dim, int norm, float p, int io_dtype, int h_dtype) {
  if (rows < 0 || dim < 1) return SSM_ERR_SHAPE;
  if (!io_type(io_dtype) || !io_type(h_dtype)) return SSM_ERR_DTYPE;
  if (io_dtype == SSM_F32 && h_dtype != SSM_F32) return SSM_ERR_DTYPE;
  if (norm != SSM_NORM_LAYER && norm != SSM_NORM_RMS) return SSM_ERR_FLAG;
  if (!(p >= 0.0f && p < 1.0f)) return SSM_ERR_FLAG;
  if (!product_fits({rows, dim})) return SSM_ERR_SHAPE;
  return dim > ssm66::add_norm::kMostDim ? SSM_ERR_UNSUPPORTED : SSM_OK;
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
  const size_t need = ssm66::gated_scan::workspace_bytes(batch, seqlen, dim, false, false);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  // several blocks read h0, and two tiles read the channels that both have
  const size_t io = (size_t)(batch * seqlen * dim) * width(io_dtype), row = (size_t)(batch * dim) * 4;
  if (!apart({{y, io}, {last_state, row}, {states, row * kept_states(seqlen)}, {workspace, need}},
             {{x, io}, {r, io}, {i, io}, {decay, (size_t)dim * 4}, {h0, row},
              {seq_lens, (size_t)batch * 4}, {reset, (size_t)(batch * seqlen)}}))
    return SSM_ERR_FLAG;
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
  const size_t need = batch == 0 ? 0
      : ssm66::gated_scan::workspace_bytes(batch, seqlen, dim, true, ddecay != nullptr);
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  const size_t io = (size_t)(batch * seqlen * dim) * width(io_dtype), row = (size_t)(batch * dim) * 4;
  if (!apart({{dx, io}, {dr, io}, {di, io}, {ddecay, (size_t)dim * 4}, {dh0, row}, {workspace, need}},
             {{x, io}, {r, io}, {i, io}, {decay, (size_t)dim * 4}, {states, row * kept_states(seqlen)},
              {seq_lens, (size_t)batch * 4}, {reset, (size_t)(batch * seqlen)}, {dy, io}, {dlast, row}}))
    return SSM_ERR_FLAG;
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
  const size_t io = (size_t)(batch * dim) * width(io_dtype);
  const Span out = {y, io}, sx = {x, io}, sr = {r, io}, si = {i, io}, sd = {decay, (size_t)dim * 4};
  if (!apart({{state, (size_t)(batch * dim) * 4}}, {out, sx, sr, si, sd}) || meet(out, sd) ||
      !apart_or_over(out, sx) || !apart_or_over(out, sr) || !apart_or_over(out, si))
    return SSM_ERR_FLAG;
  ssm66::gated_scan::StepArgs a;
  a.state = state; a.x = x; a.r = r; a.i = i; a.decay = decay; a.y = y; a.batch = batch; a.dim = (int)dim;
  return status(ssm66::gated_scan::step(a, io_dtype == SSM_F32, (hipStream_t)stream));
}

int ssm_dropout(const void* x, const void* residual, const int64_t* rng, int64_t site, float p,
                void* y, int64_t n, int io_dtype, int out_dtype, void* stream) {
  if (n < 0 || !product_fits({n})) return SSM_ERR_SHAPE;
  if (!io_type(io_dtype) || !io_type(out_dtype)) return SSM_ERR_DTYPE;
  if (!(p >= 0.0f && p < 1.0f)) return SSM_ERR_FLAG;
  if (n == 0) return SSM_OK;
  if (!x || !y || (p > 0.0f && !rng)) return SSM_ERR_NULL;
  if (!aligned(x, width(io_dtype)) || !aligned_all(width(out_dtype), {residual, y}) || !aligned(rng, 8))
    return SSM_ERR_ALIGN;
  // (in place of the other type a value would be written before its neighbours are read)
  const Span out = {y, (size_t)n * width(out_dtype)};
  if (!apart_or_over(out, {x, (size_t)n * width(io_dtype)}) || !apart_or_over(out, {residual, out.bytes}) ||
      meet(out, {rng, 16}))
    return SSM_ERR_FLAG;
  ssm66::dropout::Args a;
  a.x = x; a.residual = residual; a.y = y; a.n = n; a.drop = ssm66::drop_of(p, rng, site);
  return status(ssm66::dropout::run(a, io_dtype == SSM_F32, out_dtype == SSM_F32, (hipStream_t)stream));
}

int ssm_add_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                     int norm, float eps, float p, const int64_t* rng, int64_t site, void* y,
                     void* h, float* mean, float* rstd, int64_t rows, int64_t dim, int io_dtype,
                     int h_dtype, void* stream) {
  const int st = norm_args(rows, dim, norm, p, io_dtype, h_dtype);
  if (st != SSM_OK) return st;
  if (rows == 0) return SSM_OK;
  if (!x || !y || (p > 0.0f && !rng)) return SSM_ERR_NULL;
  if (!aligned_all(width(io_dtype), {x, y}) || !aligned_all(width(h_dtype), {residual, h}) ||
      !aligned_all(4, {weight, bias, mean, rstd}) || !aligned(rng, 8))
    return SSM_ERR_ALIGN;
  const size_t n = (size_t)(rows * dim), row = (size_t)rows * 4, col = (size_t)dim * 4;
  const Span sx = {x, n * width(io_dtype)}, sy = {y, sx.bytes}, sres = {residual, n * width(h_dtype)};
  const Span sh = {h, sres.bytes}, sw = {weight, col}, sb = {bias, col}, sg = {rng, 16};
  const Span smean = {norm == SSM_NORM_LAYER ? mean : nullptr, row}, srstd = {rstd, row};
  if (!apart({sy, sh}, {sw, sb, sg}) || !apart({smean, srstd}, {sx, sres, sy, sh, sw, sb, sg}) ||
      !apart_or_over(sy, sx) || meet(sy, sres) || !apart_or_over(sh, sres) || !apart_or_over(sh, sx))
    return SSM_ERR_FLAG;
  ssm66::add_norm::Args a = {};
  a.x = x; a.residual = residual; a.weight = weight; a.bias = bias; a.y = y; a.h = h;
  a.mean = mean; a.rstd = rstd; a.drop = ssm66::drop_of(p, rng, site);
  a.rows = rows; a.dim = (int)dim; a.rms = norm == SSM_NORM_RMS; a.eps = eps;
  return status(ssm66::add_norm::forward(a, io_dtype == SSM_F32, h_dtype == SSM_F32, (hipStream_t)stream));
}

size_t ssm_add_norm_workspace_size(int64_t rows, int64_t dim) {
  if (norm_args(rows, dim, SSM_NORM_LAYER, 0.0f, SSM_F32, SSM_F32) != SSM_OK) return 0;
  return ssm66::add_norm::workspace_bytes(rows, dim);
}

int ssm_add_norm_bwd(const void* h, const void* dy, const void* dh, const float* weight, int norm,
                     const float* mean, const float* rstd, float p, const int64_t* rng,
                     int64_t site, void* dx, void* dresidual, float* dweight, float* dbias,
                     void* workspace, size_t workspace_bytes, int64_t rows, int64_t dim,
                     int io_dtype, int h_dtype, void* stream) {
  const int st = norm_args(rows, dim, norm, p, io_dtype, h_dtype);
  if (st != SSM_OK) return st;
  if (rows > 0 && (!h || !dy || !dx || !rstd || (norm == SSM_NORM_LAYER && !mean) || (p > 0.0f && !rng)))
    return SSM_ERR_NULL;
  if (!aligned_all(width(io_dtype), {dy, dx}) || !aligned_all(width(h_dtype), {h, dh, dresidual}) ||
      !aligned_all(4, {weight, mean, rstd, dweight, dbias}) || !aligned(rng, 8) || !aligned(workspace, 256))
    return SSM_ERR_ALIGN;
  const bool sums = dweight || dbias;
  const size_t need = sums ? ssm66::add_norm::workspace_bytes(rows, dim) : 0;
  if (need > 0 && !workspace) return SSM_ERR_NULL;
  if (workspace_bytes < need) return SSM_ERR_SHAPE;
  const size_t n = (size_t)(rows * dim), row = (size_t)rows * 4, col = (size_t)dim * 4;
  const Span sh = {h, n * width(h_dtype)}, sdy = {dy, n * width(io_dtype)}, sdh = {dh, sh.bytes};
  const Span sdx = {dx, sdy.bytes}, sres = {dresidual, sh.bytes};
  const Span sw = {weight, col}, smean = {norm == SSM_NORM_LAYER ? mean : nullptr, row}, srstd = {rstd, row}, sg = {rng, 16};
  if (!apart({sdx, sres}, {sh, sw, smean, srstd, sg}) ||
      !apart({{dweight, col}, {dbias, col}, {workspace, need}}, {sh, sdy, sdh, sdx, sres, sw, smean, srstd, sg}) ||
      !apart_or_over(sdx, sdy) || !apart_or_over(sdx, sdh) || !apart_or_over(sres, sdy) || !apart_or_over(sres, sdh))
    return SSM_ERR_FLAG;
  ssm66::add_norm::Args a = {};
  a.h = (void*)h; a.dy = dy; a.dh = dh; a.weight = weight; a.mean = (float*)mean; a.rstd = (float*)rstd;
  a.drop = ssm66::drop_of(p, rng, site); a.dx = dx; a.dresidual = dresidual;
  a.dweight = dweight; a.dbias = dbias; a.part = sums ? (float2*)workspace : nullptr;
  a.rows = rows; a.dim = (int)dim; a.rms = norm == SSM_NORM_RMS;
  return status(ssm66::add_norm::backward(a, io_dtype == SSM_F32, h_dtype == SSM_F32, (hipStream_t)stream));
}

int ssm_rotary(const void* q, const void* k, const float* freqs, const int32_t* positions,
               float mscale, int interleaved, int inverse, void* q_out, void* k_out, int64_t batch,
               int64_t seqlen, int64_t heads, int64_t kheads, int64_t dim, int64_t rot,
               int io_dtype, void* stream) {
  if (batch < 0 || seqlen < 0 || heads < 1 || kheads < 0 || dim < 1) return SSM_ERR_SHAPE;
  if (rot < 2 || rot % 2 != 0 || rot > dim) return SSM_ERR_SHAPE;
  if (!io_type(io_dtype)) return SSM_ERR_DTYPE;
  const int64_t most = (int64_t)1 << 20;
  if (!product_fits({batch, seqlen}) || !product_fits({batch, seqlen, heads, dim}) ||
      !product_fits({batch, seqlen, kheads, dim}))
    return SSM_ERR_SHAPE;
  if (batch == 0 || seqlen == 0) return SSM_OK;
  if (!q || !q_out || !freqs || (kheads > 0 && (!k || !k_out))) return SSM_ERR_NULL;
  if (heads > most || kheads > most || dim > most || seqlen > 0x7fffffff ||
      !ssm66::rotary::fits(batch * seqlen, (int)(heads + kheads), (int)dim))
    return SSM_ERR_UNSUPPORTED;
  if (!aligned_all(width(io_dtype), {q, k, q_out, k_out}) || !aligned_all(4, {freqs, positions}))
    return SSM_ERR_ALIGN;
  const size_t token = (size_t)dim * width(io_dtype), tokens = (size_t)(batch * seqlen);
  const Span sq = {q, tokens * heads * token}, so = {q_out, sq.bytes};
  const Span sk = {kheads > 0 ? k : nullptr, tokens * kheads * token}, sko = {kheads > 0 ? k_out : nullptr, sk.bytes};
  const Span sf = {freqs, (size_t)rot * 2}, sp = {positions, tokens * 4};
  if (!apart({so, sko}, {sf, sp}) || !apart_or_over(so, sq) || !apart_or_over(sko, sk) || meet(so, sk) || meet(sko, sq))
    return SSM_ERR_FLAG;
  ssm66::rotary::Args a = {};
  a.q = q; a.k = kheads > 0 ? k : nullptr; a.qo = q_out; a.ko = kheads > 0 ? k_out : nullptr;
  a.freqs = freqs; a.positions = positions; a.tokens = batch * seqlen; a.L = seqlen;
  a.H = (int)heads; a.Hk = (int)kheads; a.D = (int)dim; a.pairs = (int)(rot / 2);
  a.mscale = mscale; a.sign = inverse ? -1.0f : 1.0f; a.interleaved = interleaved != 0;
  return status(ssm66::rotary::run(a, io_dtype == SSM_F32, (hipStream_t)stream));
}

}  // extern "C"
