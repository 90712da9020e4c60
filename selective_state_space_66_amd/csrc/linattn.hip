// linattn.hip -- linear attention with a decay for each head: how its walks
// (linattn_walk.h) are laid out, the sums over heads that share keys, and the
// single-token step.
#include "linattn_launch.h"
#include "ssm_device.h"

namespace ssm66 {
namespace linattn {

Tile walk_tile(bool f32, int K, int V, bool dg) {
  Tile t;
  t.KP = K <= 64 ? 64 : (K <= 128 ? 128 : 256);
  if (f32) t.VB = t.KP == 256 ? 16 : 32;
  else t.VB = (t.KP == 256 || V <= 32 || (dg && t.KP == 128)) ? 32 : 64;
  return t;
}

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// A walk's spans: blocks of one (entry, head, column slice) each, cut along
// the tokens when there are too few of them to fill the 256 CUs.
struct Spans { int n, chunks; };
Spans spans_for(int64_t blocks, int64_t L) {
  const int64_t nc = (L + kChunk - 1) / kChunk;
  int64_t n = 1;
  if (blocks > 0 && blocks < 256) {
    n = (512 + blocks - 1) / blocks;
    if (n > nc / 4) n = nc / 4;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
  }
  Spans s;
  s.chunks = nc == 0 ? 1 : (int)((nc + n - 1) / n);
  s.n = nc == 0 ? 1 : (int)((nc + s.chunks - 1) / s.chunks);
  return s;
}

struct Walk {
  Tile tile;
  Spans spans;
  int nsl;
  size_t state_bytes, cut_bytes, part_bytes;
};
Walk plan(const Problem& p, int K, int V, bool dg) {
  Walk w;
  w.tile = walk_tile(p.f32, K, V, dg);
  w.nsl = (V + w.tile.VB - 1) / w.tile.VB;
  w.spans = spans_for(p.batch * p.H * w.nsl, p.L);
  const size_t m = (size_t)(w.spans.n - 1);
  w.state_bytes = up256(m * p.batch * p.H * (dg ? 2 : 1) * (size_t)K * V * 4);
  w.cut_bytes = up256(m * p.batch * 4);
  w.part_bytes = dg ? up256((size_t)p.H * p.batch * w.nsl * w.spans.n * 4) : 0;
  return w;
}

size_t most(size_t a, size_t b) { return a > b ? a : b; }

// The parts of a backward workspace.
struct BwdLayout {
  Walk q, k, v;
  size_t states, cuts, parts, shared, total;
};
BwdLayout bwd_layout(const Problem& p, bool dg) {
  BwdLayout l;
  l.q = plan(p, p.Dv, p.Dk, dg);
  l.k = plan(p, p.Dv, p.Dk, false);
  l.v = plan(p, p.Dk, p.Dv, false);
  l.states = most(l.q.state_bytes, most(l.k.state_bytes, l.v.state_bytes));
  l.cuts = most(l.q.cut_bytes, most(l.k.cut_bytes, l.v.cut_bytes));
  l.parts = l.q.part_bytes;
  l.shared = p.H != p.Hk ? up256((size_t)p.batch * p.L * p.H * p.Dk * 4) : 0;
  l.total = l.states + l.cuts + l.parts + l.shared;
  return l;
}

hipError_t run_walk(WalkArgs a, const Problem& p, const Walk& w, bool rev, bool dg,
                    hipStream_t stream) {
  a.nspan = w.spans.n;
  a.span_chunks = w.spans.chunks;
  for (int state = w.spans.n > 1 ? 1 : 0; state >= 0; --state) {
    const hipError_t e = p.f32 ? walk_f32(a, w.tile, rev, dg, state != 0, stream)
                               : walk_bf16(a, w.tile, rev, dg, state != 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

WalkArgs walk_args(const Problem& p, char* ws, size_t cuts_at) {
  WalkArgs a = {};
  a.ws = (float*)ws;
  a.span_cut = (int32_t*)(ws + cuts_at);
  a.log_decay = p.log_decay;
  a.seq_lens = p.seq_lens;
  a.reset = p.reset;
  a.batch = p.batch;
  a.L = p.L;
  a.H = p.H;
  return a;
}

// dq and dk of keys shared by `rep` heads: the heads' fp32 parts added in
// order, rounded once.  Four columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void sum_heads_kernel(const float* part, T* out, int64_t n4, int Hk,
                                                        int rep, int D4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const int64_t row = i / ((int64_t)Hk * D4);
  const int rest = (int)(i - row * Hk * D4), g = rest / D4, d = rest - g * D4;
  const float4* src = (const float4*)part + (row * Hk + g) * (int64_t)rep * D4 + d;
  float4 s = src[0];
  for (int r = 1; r < rep; ++r) {
    const float4 x = src[(int64_t)r * D4];
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  if constexpr (sizeof(T) == 4) {
    ((float4*)out)[i] = s;
  } else {
    uint2 v;
    v.x = pack_bf16x2(s.x, s.y);
    v.y = pack_bf16x2(s.z, s.w);
    ((uint2*)out)[i] = v;
  }
}

hipError_t sum_heads(const Problem& p, const float* part, void* out, hipStream_t stream) {
  const int64_t n4 = p.batch * p.L * p.Hk * (p.Dk / 4);
  if (n4 == 0) return hipSuccess;
  const dim3 grid((uint32_t)((n4 + 255) / 256));
  if (p.f32)
    sum_heads_kernel<float><<<grid, 256, 0, stream>>>(part, (float*)out, n4, p.Hk, p.H / p.Hk, p.Dk / 4);
  else
    sum_heads_kernel<bf16_bits><<<grid, 256, 0, stream>>>(part, (bf16_bits*)out, n4, p.Hk, p.H / p.Hk, p.Dk / 4);
  return hipGetLastError();
}

// the gradient of each head's log-decay: its blocks' sums, in a fixed order
__global__ __launch_bounds__(64) void sum_parts_kernel(const float* part, float* out, int64_t n) {
  const float* src = part + (int64_t)blockIdx.x * n;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 64) s += (double)src[i];
  __shared__ double all[64];
  all[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
    for (int i = 0; i < 64; ++i) t += all[i];
    out[blockIdx.x] = (float)t;
  }
}

}  // namespace

size_t fwd_workspace(const Problem& p) {
  const Walk w = plan(p, p.Dk, p.Dv, false);
  return w.state_bytes + w.cut_bytes;
}

size_t bwd_workspace(const Problem& p, bool dg) { return bwd_layout(p, dg).total; }

hipError_t forward(const Problem& p, const FwdOut& o, void* workspace, hipStream_t stream) {
  const Walk w = plan(p, p.Dk, p.Dv, false);
  WalkArgs a = walk_args(p, (char*)workspace, w.state_bytes);
  a.a = p.q; a.b = p.k; a.c = p.v; a.out = o.o;
  a.Ha = p.Hk; a.Hb = p.Hk; a.Hc = p.H;
  a.K = p.Dk; a.V = p.Dv;
  a.init = p.h0; a.state_sv = p.Dk; a.state_sk = 1;
  a.final_state = o.last_state;
  a.s_intra = p.scale; a.s_state = 1.0f; a.s_inter = p.scale;
  return run_walk(a, p, w, false, false, stream);
}

hipError_t backward(const Problem& p, const BwdArgs& g, void* workspace, hipStream_t stream) {
  const bool dg = g.dlog_decay != nullptr;
  const BwdLayout l = bwd_layout(p, dg);
  char* const ws = (char*)workspace;
  float* const parts = (float*)(ws + l.states + l.cuts);
  float* const shared = (float*)(ws + l.states + l.cuts + l.parts);
  const WalkArgs common = walk_args(p, ws, l.states);
  hipError_t e;
  {  // dq, and the log-decay's gradient
    WalkArgs a = common;
    a.a = g.dout; a.b = p.v; a.c = p.k; a.x = p.q;
    a.Ha = p.H; a.Hb = p.H; a.Hc = p.Hk;
    a.K = p.Dv; a.V = p.Dk;
    a.out = l.shared ? (void*)shared : g.dq;
    a.out_f32 = l.shared != 0;
    a.init = p.h0; a.state_sv = 1; a.state_sk = p.Dk;
    a.dlast = g.dlast;
    a.dg_part = parts;
    a.s_intra = p.scale; a.s_state = 1.0f; a.s_inter = p.scale;
    if ((e = run_walk(a, p, l.q, false, dg, stream)) != hipSuccess) return e;
    if (l.shared && (e = sum_heads(p, shared, g.dq, stream)) != hipSuccess) return e;
    if (dg) {
      sum_parts_kernel<<<dim3((uint32_t)p.H), 64, 0, stream>>>(parts, g.dlog_decay,
                                                               p.batch * l.q.nsl * l.q.spans.n);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  WalkArgs a = common;
  a.init = g.dlast;
  a.s_intra = p.scale; a.s_state = p.scale; a.s_inter = 1.0f;
  {  // dv and the initial state's gradient
    a.a = p.k; a.b = p.q; a.c = g.dout; a.out = g.dv;
    a.Ha = p.Hk; a.Hb = p.Hk; a.Hc = p.H;
    a.K = p.Dk; a.V = p.Dv;
    a.state_sv = p.Dk; a.state_sk = 1;
    a.final_state = g.dh0;
    if ((e = run_walk(a, p, l.v, true, false, stream)) != hipSuccess) return e;
  }
  {  // dk
    a.a = p.v; a.b = g.dout; a.c = p.q;
    a.out = l.shared ? (void*)shared : g.dk;
    a.out_f32 = l.shared != 0;
    a.Ha = p.H; a.Hb = p.H; a.Hc = p.Hk;
    a.K = p.Dv; a.V = p.Dk;
    a.state_sv = 1; a.state_sk = p.Dk;
    a.final_state = nullptr;
    if ((e = run_walk(a, p, l.k, true, false, stream)) != hipSuccess) return e;
    if (l.shared && (e = sum_heads(p, shared, g.dk, stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---- one token ----------------------------------------------------------------
//
// state = lam state + v k^T, o = scale state q, per head.  Reads and writes the
// fp32 state once (8 bytes per element) and little else, so HBM bounds it.
// LPR lanes (a power of two) share a row of Dk states, four each; a wave holds
// 64 / LPR rows at a time and R such sets, all loaded before the first is used.
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;

template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *(const f32x4*)p;
  } else {
    const uint2 v = *(const uint2*)p;
    return f32x4{__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                 __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
  }
}

template <typename T, int LPR, int R>
__global__ __launch_bounds__(256) void linattn_step_kernel(const StepArgs p, int nb) {
  constexpr int kRows = 64 / LPR;  // rows of a wave's load
  const uint32_t bh = blockIdx.x / (uint32_t)nb, part = blockIdx.x % (uint32_t)nb;
  const uint32_t b = bh / (uint32_t)p.H, h = bh - b * (uint32_t)p.H;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = 4 * (lane % LPR);
  const int v0 = ((int)part * 4 + w) * (kRows * R) + lane / LPR;
  const int Dk = p.Dk, Dv = p.Dv;
  const bool in = col < Dk;
  float* const st = p.state + (int64_t)bh * Dk * Dv + col;
  f32x4 s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int v = v0 + r * kRows;
    s[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (in && v < Dv) s[r] = __builtin_nontemporal_load((const f32x4*)(st + (int64_t)v * Dk));
  }
  const int64_t kv = (int64_t)b * p.Hk + h / (uint32_t)(p.H / p.Hk);
  f32x4 q = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, k = q;
  if (in) {
    q = load4((const T*)p.q + kv * Dk + col);
    k = load4((const T*)p.k + kv * Dk + col);
  }
  const float lam = exp2_hw(p.log_decay[h] * kLog2e);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int v = v0 + r * kRows;
    if (v >= Dv) continue;  // the same for all lanes of a row
    const float x = to_f32(((const T*)p.v)[(int64_t)bh * Dv + v]);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[r][i] = fmaf(lam, s[r][i], x * k[i]);
      dot = fmaf(s[r][i], q[i], dot);
    }
    if (in) __builtin_nontemporal_store(s[r], (f32x4*)(st + (int64_t)v * Dk));
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) dot += __shfl_xor(dot, m);
    if (lane % LPR == 0) store_io((T*)p.o + (int64_t)bh * Dv + v, p.scale * dot);
  }
}

template <typename T, int LPR>
hipError_t step_rows(const StepArgs& a, hipStream_t stream) {
  // four sets of rows in flight per wave once there are enough rows for it
  const int64_t heads = a.batch * a.H;
  const int rows = 64 / LPR * 4;
  const bool many = heads * ((a.Dv + rows - 1) / rows) >= 4096;
  const int per = many ? 4 * rows : rows;
  const int nb = (a.Dv + per - 1) / per;
  const int64_t n = heads * nb;
  if (n > 0x7fffffff) return hipErrorInvalidValue;
  const dim3 grid((uint32_t)n);
  if (many) linattn_step_kernel<T, LPR, 4><<<grid, 256, 0, stream>>>(a, nb);
  else linattn_step_kernel<T, LPR, 1><<<grid, 256, 0, stream>>>(a, nb);
  return hipGetLastError();
}

template <typename T>
hipError_t step_typed(const StepArgs& a, hipStream_t stream) {
  const int need = a.Dk / 4;
  if (need <= 4) return step_rows<T, 4>(a, stream);
  if (need <= 8) return step_rows<T, 8>(a, stream);
  if (need <= 16) return step_rows<T, 16>(a, stream);
  if (need <= 32) return step_rows<T, 32>(a, stream);
  return step_rows<T, 64>(a, stream);
}

}  // namespace

hipError_t step(const StepArgs& a, hipStream_t stream) {
  return a.f32 ? step_typed<float>(a, stream) : step_typed<bf16_bits>(a, stream);
}

}  // namespace linattn
}  // namespace ssm66
