// linattn.hip -- linear attention with a decay for each head: how its walks
// (linattn_walk.h) are laid out, the sums over heads that share keys, and the
// single-token step.
#include "linattn_launch.h"
#include "lm_grid.h"
#include "ssm_device.h"

namespace ssm66 {
namespace linattn {

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Pieces of a cut walk, each a state that the spans behind it read and add: one
// head of 64 x 64 over 32768 tokens takes 62.5 us in 65 spans, 79 in 128 and 73 in
// 33; forwards and backwards 275, 334 and 330.
constexpr int kMostPieces = 64;

int64_t chunks_of(int64_t L) { return (L + kChunk - 1) / kChunk; }

// Row widths that a kernel is made for.  Only fp32 rows have one of 96, where
// all of a chunk's work grows with the width.
int padded(int K, bool f32) { return K <= 64 ? 64 : (f32 && K <= 96 ? 96 : (K <= 128 ? 128 : 256)); }

// How a walk is laid out.
//
// Tile.  A block takes 64 columns where its CU is its own (bf16 rows of up to
// 128; 2048 tokens: 77 us against 83 with 32 for 192 (entry, head) pairs of 64
// columns, 128 keys, 134 against 153 for 512 pairs, 64 keys), but 32, two blocks
// to a CU, where 64 would leave half of the second round of blocks empty or more
// (97 against 114 us for 192 pairs of 128 columns, 64 keys; 150 against 160 with
// 128 keys).  fp32 rows and the walk with the log-decay's gradient have three
// parts of most operands and take 32, fp32 rows of 256 take 16.
//
// Spans.  Too few blocks for one round are cut along the tokens as often as
// fills it; each span then needs the state before it, from a walk that reads b
// and c once more (1 x 65536 x 16 heads of 128: 8 spans, 370 us and 152 us for
// the states).  Cutting two thirds of a round costs more than it gives (94 + 27
// against 87 us for the 192 pairs above), and so do sequences under 16 chunks.
struct Walk {
  Tile tile, state_tile;
  int nsl, nspan, span_chunks, pieces, piece_chunks;
  size_t state_bytes, cut_bytes, part_bytes;
};
Walk plan(const Problem& p, int K, int V, bool dg) {
  Walk w;
  const int KP = padded(K, p.f32);
  const int64_t pairs = p.batch * p.H;
  const int64_t n64 = pairs * ((V + 63) / 64);
  w.tile.KP = w.state_tile.KP = KP;
  if (p.f32) w.tile.VB = KP == 256 ? 16 : 32;
  else w.tile.VB = !dg && KP <= 128 && V > 32 && (n64 <= 256 || n64 > 384) ? 64 : 32;
  w.nsl = (V + w.tile.VB - 1) / w.tile.VB;
  const int64_t blocks = pairs * w.nsl;
  const int64_t round = !p.f32 && !dg && KP <= 128 && w.tile.VB == 32 ? 512 : 256;
  const int64_t nc = chunks_of(p.L);
  int64_t spans = blocks > 0 && nc >= 16 ? round / blocks : 1;
  if (spans > nc / 4) spans = nc / 4;
  if (spans > kMostPieces + 1) spans = kMostPieces + 1;
  if (spans < 1) spans = 1;
  // pieces for the state walk: about 512 blocks of it, four chunks at least
  w.state_tile.VB = p.f32 || KP == 256 ? w.tile.VB : (V > 64 && !dg ? 128 : (V > 32 && !(dg && KP == 128) ? 64 : 32));
  const int64_t state_blocks = pairs * ((V + w.state_tile.VB - 1) / w.state_tile.VB);
  int64_t per = (nc + spans - 1) / spans;  // chunks of a span
  int64_t split = 1;                       // pieces of a span
  if (spans > 1) {
    split = 512 / (state_blocks * (spans - 1));
    if (split > per / 4) split = per / 4;
    if (split > kMostPieces / (spans - 1)) split = kMostPieces / (spans - 1);
    if (split < 1) split = 1;
    per = (per + split - 1) / split * split;
  }
  if (per < 1) per = 1;
  w.span_chunks = (int)per;
  w.piece_chunks = (int)(per / split);
  w.nspan = nc == 0 ? 1 : (int)((nc + per - 1) / per);
  w.pieces = (int)((w.nspan - 1) * split);
  w.state_bytes = up256((size_t)w.pieces * pairs * (dg ? 2 : 1) * (size_t)K * V * 4);
  w.cut_bytes = up256((size_t)w.pieces * p.batch * 4);
  w.part_bytes = dg ? up256((size_t)pairs * w.nsl * w.nspan * 8) : 0;
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
  a.nspan = w.nspan;
  a.span_chunks = w.span_chunks;
  a.pieces = w.pieces;
  a.piece_chunks = w.piece_chunks;
  for (int state = w.pieces > 0 ? 1 : 0; state >= 0; --state) {
    const Tile t = state ? w.state_tile : w.tile;
    const hipError_t e = p.f32 ? walk_f32(a, t, rev, dg, state != 0, stream)
                               : walk_bf16(a, t, rev, dg, state != 0, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

WalkArgs walk_args(const Problem& p, char* ws, size_t cuts_at) {
  WalkArgs a = {};
  a.ws = (float*)ws;
  a.piece_cut = (int32_t*)(ws + cuts_at);
  a.log_decay = p.log_decay;
  a.seq_lens = p.seq_lens;
  a.reset = p.reset;
  a.batch = p.batch;
  a.L = p.L;
  a.H = p.H;
  return a;
}

// dq and dk of keys shared by `rep` heads: the heads' fp32 parts added in
// order, rounded once.  Four columns per thread; HBM or caches bound it (5.4 us
// for 3 x 1537 x 12 heads of 72, 4 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void sum_heads_kernel(const float* part, T* out, int64_t n4, int Hk,
                                                        int rep, int D4) {
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
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
  const Grid g = grid_of((n4 + 255) / 256, 256);
  const dim3 grid(g.x, g.more);
  if (p.f32)
    sum_heads_kernel<float><<<grid, 256, 0, stream>>>(part, (float*)out, n4, p.Hk, p.H / p.Hk, p.Dk / 4);
  else
    sum_heads_kernel<bf16_bits><<<grid, 256, 0, stream>>>(part, (bf16_bits*)out, n4, p.Hk, p.H / p.Hk, p.Dk / 4);
  return hipGetLastError();
}

// the gradient of each head's log-decay: its blocks' sums, in a fixed order, in
// fp64 (a few hundred numbers: 5 us, of which a launch is 4)
__global__ __launch_bounds__(64) void sum_parts_kernel(const double* part, float* out, int64_t n) {
  const double* src = part + (int64_t)blockIdx.x * n;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 64) s += src[i];
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
  double* const parts = (double*)(ws + l.states + l.cuts);
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
                                                               p.batch * l.q.nsl * l.q.nspan);
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
// fp32 state once (8 bytes per element) and little else, so HBM bounds it: 256
// sequences of 24 heads, 64 x 128, take 68.7 us, 5.95 TB/s (the part of the
// states that the Infinity Cache still holds is read from there).  One sequence
// of 16 heads of 64 takes 2.8 us, a launch.
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
  const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x;  // y: more blocks than x holds
  const uint32_t bh = id / (uint32_t)nb, part = id % (uint32_t)nb;
  if (bh >= (uint32_t)(p.batch * p.H)) return;
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
  const Grid g = grid_of(n, 256);
  const dim3 grid(g.x, g.more);
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
