// group_norm.hip -- group norm over channels-last tensors with an activation
// and a gate, forward and backward.
//
// x (batch, rows, C), C = groups * cg.  For entry n and group g, over the M =
// rows * cg values of the group,
//   mean = sum x / M,   rstd = 1 / sqrt(sum (x - mean)^2 / M + eps),
//   xh = (x - mean) rstd,   u = xh w_c + b_c,   a = act(u),   y = a silu(z),
// and backwards, with da = dy silu(z), du = da act'(u), dn = du w_c,
//   dx = rstd (dn - sum dn / M - xh sum(dn xh) / M),
//   dw_c = sum du xh,  db_c = sum du,  dz = dy a silu'(z).
// A few operations per value: HBM bounds all of it.
//
// Two forms.
// - One row (rows == 1: a norm of each token's heads) whose groups fit the
//   registers of a wave: a group is held by a power of two of lanes, read
//   once, its mean and the squares about it taken from registers.  A thread
//   keeps its columns for all the rows it takes, so the backward adds dw and
//   db in registers and each block writes one row of partial sums.
// - Anything else: the rows of an entry are cut into pieces.  Pass 1 takes,
//   for each channel and piece, the mean and the squares about it (from sums
//   about the thread's first value, so a large common offset costs no
//   precision); a small kernel merges them per group by the parallel form of
//   the variance; pass 2 reads x again and writes.  The backward has the same
//   two passes around the sums of du and du xh.
//
// Measured (a copy reaches 5.2 TB/s).  One row: 16384 tokens x 1536 channels in
// 24 groups with gate, bf16: forwards 33.8 us (4.5 TB/s), backwards 54.5 (4.6)
// and 4.8 for the channel sums.  Pieces: 6 x 4095 x 320 in 32 groups with silu,
// fp32: forwards 9.8 + 5.4 + 11.9 us, backwards 13.2 + 5.8 + 16.2 + 3.9; the
// passes over the tensors run at 3.2 to 5.8 TB/s (the second finds x in the
// Infinity Cache), the merges and the channel sums little above a launch.
// All sums are fp32 in a fixed order (no atomics).
#include "group_norm_launch.h"
#include "lm_grid.h"
#include "ssm_device.h"

namespace ssm66 {
namespace group_norm {

namespace {

__device__ __forceinline__ float sigmoid_f(float v) { return rcp_hw(1.0f + exp2_hw(-v * kLog2e)); }

// VEC consecutive io values as one memory access
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  struct alignas(sizeof(T) * VEC) A { T v[VEC]; };
  const A a = *(const A*)p;
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = to_f32(a.v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  struct alignas(sizeof(T) * VEC) A { T v[VEC]; };
  A a;
#pragma unroll
  for (int i = 0; i < VEC; ++i) store_io(&a.v[i], f[i]);
  *(A*)p = a;
}

// What one value needs forwards and backwards.
template <bool SILU, bool GATE>
struct Point {
  static __device__ __forceinline__ float forward(float u, float z) {
    const float a = SILU ? u * sigmoid_f(u) : u;
    return GATE ? a * silu_f(z) : a;
  }
  // du from dy, and dz
  static __device__ __forceinline__ float backward(float u, float z, float dy, float* dz) {
    float a = u, da = 1.0f;
    if (SILU) {
      const float s = sigmoid_f(u);
      a = u * s;
      da = s * (1.0f + u * (1.0f - s));
    }
    if (GATE) {
      const float s = sigmoid_f(z);
      *dz = dy * a * (s * (1.0f + z * (1.0f - s)));
      dy *= z * s;
    }
    return dy * da;
  }
};

// sum over the LPG lanes that share a group
template <int LPG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = LPG / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// ---- one row per entry --------------------------------------------------------
//
// The slots of a row are groups x LPG lanes; a lane holds NV vectors of VEC
// channels, LPG vectors apart.  A block takes `tile` slots (blockIdx.y) and
// 256 / tile rows at a time.

template <typename T, int VEC, int LPG, int NV, bool SILU, bool GATE>
__global__ __launch_bounds__(256) void rows_fwd_kernel(const Args p, int tile, int rpb) {
  const int slot = blockIdx.y * tile + (int)threadIdx.x % tile;
  const int r0 = (int)threadIdx.x / tile;
  const int g = slot / LPG, l = slot % LPG;
  if (r0 >= rpb || g >= p.groups) return;  // whole groups of lanes leave
  const int cg = p.C / p.groups;
  const float inv = 1.0f / (float)cg;
  const T* const x = (const T*)p.x;
  const T* const z = (const T*)p.z;
  float w[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (l + j * LPG) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[j][i] = p.weight && c < cg ? p.weight[g * cg + c + i] : 1.0f;
      b[j][i] = p.bias && c < cg ? p.bias[g * cg + c + i] : 0.0f;
    }
  }
  for (int64_t n = (int64_t)blockIdx.x * rpb + r0; n < p.batch; n += (int64_t)gridDim.x * rpb) {
    const int64_t at = n * p.C + g * cg;
    float v[NV][VEC], gz[NV][VEC];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (l + j * LPG) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = gz[j][i] = 0.0f;
      if (c < cg) {
        load_vec<T, VEC>(x + at + c, v[j]);
        if (GATE) load_vec<T, VEC>(z + at + c, gz[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s += v[j][i];
    // the mean, and what its rounding left (a common offset is large beside it);
    // then the squares about both (those about the first part alone less the
    // second's square can fall below zero where little varies)
    const float m0 = group_sum<LPG>(s) * inv;
    float q = 0.0f, left = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (l + j * LPG) * VEC < cg;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = in ? v[j][i] - m0 : 0.0f;
        left += v[j][i];
      }
    }
    left = group_sum<LPG>(left) * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool in = (l + j * LPG) * VEC < cg;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j][i] = in ? v[j][i] - left : 0.0f;
        q = fmaf(v[j][i], v[j][i], q);
      }
    }
    const float mean = m0 + left;
    const float rstd = 1.0f / sqrtf(fmaf(group_sum<LPG>(q), inv, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (l + j * LPG) * VEC;
      float y[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        y[i] = Point<SILU, GATE>::forward(fmaf(v[j][i] * rstd, w[j][i], b[j][i]), gz[j][i]);
      if (c < cg) store_vec<T, VEC>((T*)p.y + at + c, y);
    }
    if (l == 0) {
      if (p.mean) p.mean[n * p.groups + g] = mean;
      if (p.rstd) p.rstd[n * p.groups + g] = rstd;
    }
  }
}

template <typename T, int VEC, int LPG, int NV, bool SILU, bool GATE>
__global__ __launch_bounds__(256) void rows_bwd_kernel(const Args p, int tile, int rpb) {
  const int slot = blockIdx.y * tile + (int)threadIdx.x % tile;
  const int r0 = (int)threadIdx.x / tile;
  const int g = slot / LPG, l = slot % LPG;
  const bool here = r0 < rpb && g < p.groups;
  const int cg = p.C / p.groups;
  const float inv = 1.0f / (float)cg;
  float w[NV][VEC], b[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (l + j * LPG) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[j][i] = p.weight && here && c < cg ? p.weight[g * cg + c + i] : 1.0f;
      b[j][i] = p.bias && here && c < cg ? p.bias[g * cg + c + i] : 0.0f;
      dw[j][i] = db[j][i] = 0.0f;
    }
  }
  if (here) {
    for (int64_t n = (int64_t)blockIdx.x * rpb + r0; n < p.batch; n += (int64_t)gridDim.x * rpb) {
      const int64_t at = n * p.C + g * cg;
      float v[NV][VEC], gz[NV][VEC], dy[NV][VEC];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (l + j * LPG) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = gz[j][i] = dy[j][i] = 0.0f;
        if (c < cg) {
          load_vec<T, VEC>((const T*)p.x + at + c, v[j]);
          load_vec<T, VEC>((const T*)p.dy + at + c, dy[j]);
          if (GATE) load_vec<T, VEC>((const T*)p.z + at + c, gz[j]);
        }
      }
      const float mean = p.mean[n * p.groups + g], rstd = p.rstd[n * p.groups + g];
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool in = (l + j * LPG) * VEC < cg;
        float dz[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = in ? (v[j][i] - mean) * rstd : 0.0f;
          const float du =
              Point<SILU, GATE>::backward(fmaf(xh, w[j][i], b[j][i]), gz[j][i], dy[j][i], &dz[i]);
          dw[j][i] = fmaf(du, xh, dw[j][i]);
          db[j][i] += du;
          v[j][i] = xh;
          dy[j][i] = in ? du * w[j][i] : 0.0f;
          s1 += dy[j][i];
          s2 = fmaf(dy[j][i], xh, s2);
        }
        if (GATE && in) store_vec<T, VEC>((T*)p.dz + at + (l + j * LPG) * VEC, dz);
      }
      s1 = group_sum<LPG>(s1) * inv;
      s2 = group_sum<LPG>(s2) * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float dx[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) dx[i] = rstd * (dy[j][i] - s1 - v[j][i] * s2);
        const int c = (l + j * LPG) * VEC;
        if (c < cg) store_vec<T, VEC>((T*)p.dx + at + c, dx);
      }
    }
  }
  if (!p.dweight && !p.dbias) return;
  // the block's rows added in order, then one row of partial sums
  __shared__ float2 sums[256];
  float2* const part = (float2*)p.ws + (int64_t)blockIdx.x * p.C;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = (l + j * LPG) * VEC + i;
      float2 t = make_float2(db[j][i], dw[j][i]);
      if (rpb > 1) {
        __syncthreads();
        sums[threadIdx.x] = t;
        __syncthreads();
        if (r0 == 0)
          for (int r = 1; r < rpb; ++r) {
            const float2 o = sums[threadIdx.x + r * tile];
            t.x += o.x;
            t.y += o.y;
          }
      }
      if (here && r0 == 0 && c < cg) part[g * cg + c] = t;
    }
}

// ---- any number of rows -------------------------------------------------------
//
// A block takes `tile` vector columns (blockIdx.y) of one piece of the rows of
// one entry (block_of() = entry * pieces + piece), 256 / tile rows at a time.

// the number of a block along x and z
__device__ __forceinline__ uint32_t block_of() { return blockIdx.z * gridDim.x + blockIdx.x; }

struct Where {
  uint32_t block;
  int64_t n, row0, row1;
  int r0, col;
  bool here;
};
template <int VEC>
__device__ __forceinline__ Where where(const Args& p, int tile, int rpb) {
  Where w;
  w.block = block_of();
  w.n = w.block / (uint32_t)p.pieces;
  const int64_t piece = w.block % (uint32_t)p.pieces;
  w.row0 = piece * p.piece_rows;
  w.row1 = w.row0 + p.piece_rows < p.rows ? w.row0 + p.piece_rows : p.rows;
  w.r0 = (int)threadIdx.x / tile;
  w.col = (blockIdx.y * tile + (int)threadIdx.x % tile) * VEC;
  w.here = w.r0 < rpb && w.col < p.C;
  return w;
}

// What a thread reads of a row.
template <int VEC>
struct Row { float x[VEC], z[VEC], dy[VEC]; };

// One thread's rows, U of them loaded before the first is used: the pieces are
// short and few blocks share a CU, so a row at a time waits for memory each time.
template <int U, typename Load, typename Use, typename V>
__device__ __forceinline__ void rows_ahead(const Where& w, int rpb, Load load, Use use, V (&v)[U]) {
  int64_t r = w.row0 + w.r0;
  for (; r + (int64_t)(U - 1) * rpb < w.row1; r += (int64_t)U * rpb) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(r + (int64_t)u * rpb, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) use(r + (int64_t)u * rpb, v[u]);
  }
  for (; r < w.row1; r += rpb) {
    load(r, v[0]);
    use(r, v[0]);
  }
}

// (count, mean, sum of squares about it) of two disjoint sets of values
struct Moments { float n, mean, m2; };
__device__ __forceinline__ Moments merge(Moments a, Moments b) {
  const float n = a.n + b.n;
  if (n == 0.0f) return a;
  const float d = b.mean - a.mean, f = b.n / n;
  return Moments{n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}

template <typename T, int VEC>
__global__ __launch_bounds__(256) void piece_stats_kernel(const Args p, int tile, int rpb) {
  const Where w = where<VEC>(p, tile, rpb);
  if (w.n >= p.batch) return;
  const T* const x = (const T*)p.x + w.n * p.rows * p.C + w.col;
  float first[VEC], s[VEC], q[VEC];
  float cnt = 0.0f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) first[i] = s[i] = q[i] = 0.0f;
  if (w.here) {
    const int64_t r0 = w.row0 + w.r0;
    if (r0 < w.row1) load_vec<T, VEC>(x + r0 * p.C, first);
    Row<VEC> buf[4];
    rows_ahead(w, rpb, [&](int64_t r, Row<VEC>& v) { load_vec<T, VEC>(x + r * p.C, v.x); },
               [&](int64_t, const Row<VEC>& v) {
                 cnt += 1.0f;
#pragma unroll
                 for (int i = 0; i < VEC; ++i) {
                   const float d = v.x[i] - first[i];
                   s[i] += d;
                   q[i] = fmaf(d, d, q[i]);
                 }
               }, buf);
  }
  __shared__ float3 all[256];
  float2* const part = (float2*)p.ws + (int64_t)w.block * p.C;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float inv = cnt > 0.0f ? 1.0f / cnt : 0.0f;
    Moments m{cnt, fmaf(s[i], inv, first[i]), fmaxf(q[i] - s[i] * s[i] * inv, 0.0f)};
    if (q[i] != q[i]) m.m2 = q[i];  // fmaxf would lose a NaN
    if (rpb > 1) {
      __syncthreads();
      all[threadIdx.x] = make_float3(m.n, m.mean, m.m2);
      __syncthreads();
      if (w.r0 == 0)
        for (int r = 1; r < rpb; ++r) {
          const float3 o = all[threadIdx.x + r * tile];
          m = merge(m, Moments{o.x, o.y, o.z});
        }
    }
    if (w.here && w.r0 == 0) part[w.col + i] = make_float2(m.mean, m.m2);
  }
}

__device__ __forceinline__ float block_sum(float v, float* scratch) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  __syncthreads();
  if (lane == 0) scratch[w] = v;
  __syncthreads();
  return scratch[0] + scratch[1] + scratch[2] + scratch[3];
}

// What a merge takes of the partial sums: slice blockIdx.y of one group's pieces.
struct Slice {
  uint32_t group;  // entry * groups + group of the entry
  const float2* part;
  int64_t n, piece0, rows, m;  // entry, first piece, rows, partial sums (pieces x channels of the group)
  int g, cg;
};
__device__ __forceinline__ Slice slice_of(const Args& p, int slice_pieces) {
  Slice l;
  l.group = block_of();
  l.n = l.group / (uint32_t)p.groups;
  l.g = l.group % (uint32_t)p.groups;
  l.cg = p.C / p.groups;
  l.piece0 = (int64_t)blockIdx.y * slice_pieces;
  const int64_t left = p.pieces - l.piece0, pieces = left < slice_pieces ? left : slice_pieces;
  l.part = (const float2*)p.ws + (l.n * p.pieces + l.piece0) * p.C + l.g * l.cg;
  l.m = pieces * l.cg;
  const int64_t row0 = l.piece0 * p.piece_rows, row1 = row0 + pieces * p.piece_rows;
  l.rows = (row1 < p.rows ? row1 : p.rows) - row0;
  return l;
}

// One block per (entry, group) and slice: the mean and the squares about it from
// the means and squares of the channels' pieces; the group's mean and rstd where
// one slice is all, else the slice's moments for join_stats_kernel.
__global__ __launch_bounds__(256) void merge_stats_kernel(const Args p, int slice_pieces, float4* moments,
                                                          float* mean_out, float* rstd_out) {
  __shared__ float scratch[4];
  const Slice sl = slice_of(p, slice_pieces);
  if (sl.n >= p.batch) return;
  const int cg = sl.cg;
  const float2* const part = sl.part;
  const int64_t m = sl.m;
  const float total = (float)sl.rows * (float)cg;
  auto count = [&](int64_t piece) {
    const int64_t left = p.rows - (sl.piece0 + piece) * p.piece_rows;
    return (float)(left < p.piece_rows ? left : p.piece_rows);
  };
  // about the first channel's mean, so that a common offset cancels exactly;
  // a thread's first kHeld entries stay in registers for the squares
  constexpr int kHeld = 8;
  const float base = part[0].x;
  float2 held[kHeld];
  float cnt[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int64_t i = threadIdx.x + 256 * j;
    const int64_t piece = i < m ? i / cg : 0;
    held[j] = i < m ? part[piece * p.C + (i - piece * cg)] : make_float2(0.0f, 0.0f);
    cnt[j] = i < m ? count(piece) : 0.0f;
  }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) s = cnt[j] != 0.0f ? fmaf(cnt[j], held[j].x - base, s) : s;
  for (int64_t i = threadIdx.x + 256 * kHeld; i < m; i += 256) {
    const int64_t piece = i / cg;
    s = fmaf(count(piece), part[piece * p.C + (i - piece * cg)].x - base, s);
  }
  const float mean = base + block_sum(s, scratch) / total;
  float q = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const float d = held[j].x - mean;
    q = cnt[j] != 0.0f ? q + fmaf(cnt[j] * d, d, held[j].y) : q;
  }
  for (int64_t i = threadIdx.x + 256 * kHeld; i < m; i += 256) {
    const int64_t piece = i / cg;
    const float2 e = part[piece * p.C + (i - piece * cg)];
    const float d = e.x - mean;
    q += fmaf(count(piece) * d, d, e.y);
  }
  q = block_sum(q, scratch);
  if (threadIdx.x != 0) return;
  if (gridDim.y > 1) {
    moments[(int64_t)sl.group * gridDim.y + blockIdx.y] = make_float4(total, mean, q, 0.0f);
  } else {
    mean_out[sl.group] = mean;
    rstd_out[sl.group] = 1.0f / sqrtf(q / total + p.eps);
  }
}

// One thread per (entry, group): its slices in order, about the first one's mean.
__global__ __launch_bounds__(256) void join_stats_kernel(const float4* moments, int slices, int64_t n,
                                                         float eps, float* mean_out, float* rstd_out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float4* const e = moments + i * slices;
  const float base = e[0].y;
  float total = 0.0f, s = 0.0f, q = 0.0f;
  for (int k = 0; k < slices; ++k) {
    total += e[k].x;
    s = fmaf(e[k].x, e[k].y - base, s);
  }
  const float mean = base + s / total;
  for (int k = 0; k < slices; ++k) q += fmaf(e[k].x * (e[k].y - mean), e[k].y - mean, e[k].z);
  mean_out[i] = mean;
  rstd_out[i] = 1.0f / sqrtf(q / total + eps);
}

template <typename T, int VEC, bool SILU, bool GATE>
__global__ __launch_bounds__(256) void apply_fwd_kernel(const Args p, const float* mean, const float* rstd,
                                                        int tile, int rpb) {
  const Where w = where<VEC>(p, tile, rpb);
  if (!w.here || w.n >= p.batch) return;
  const int cg = p.C / p.groups;
  // y = x a + b with the norm folded into a and b would lose the mean's
  // cancellation; x - mean comes first
  float mu[VEC], sc[VEC], sh[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = w.col + i;
    const int64_t at = w.n * p.groups + c / cg;
    mu[i] = mean[at];
    sc[i] = rstd[at] * (p.weight ? p.weight[c] : 1.0f);
    sh[i] = p.bias ? p.bias[c] : 0.0f;
  }
  const int64_t base = w.n * p.rows * p.C + w.col;
  Row<VEC> buf[4];
  rows_ahead(w, rpb, [&](int64_t r, Row<VEC>& v) {
    load_vec<T, VEC>((const T*)p.x + base + r * p.C, v.x);
    if (GATE) load_vec<T, VEC>((const T*)p.z + base + r * p.C, v.z);
  }, [&](int64_t r, const Row<VEC>& v) {
    float y[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      y[i] = Point<SILU, GATE>::forward(fmaf(v.x[i] - mu[i], sc[i], sh[i]), GATE ? v.z[i] : 0.0f);
    store_vec<T, VEC>((T*)p.y + base + r * p.C, y);
  }, buf);
}

// pass 1 of the backward: per channel and piece, the sums of du and du xh
template <typename T, int VEC, bool SILU, bool GATE>
__global__ __launch_bounds__(256) void piece_grads_kernel(const Args p, int tile, int rpb) {
  const Where w = where<VEC>(p, tile, rpb);
  if (w.n >= p.batch) return;
  const int cg = p.C / p.groups;
  float mu[VEC], rs[VEC], wt[VEC], sh[VEC], s1[VEC], s2[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = w.here ? w.col + i : 0;
    const int64_t at = w.n * p.groups + c / cg;
    mu[i] = p.mean[at];
    rs[i] = p.rstd[at];
    wt[i] = p.weight ? p.weight[c] : 1.0f;
    sh[i] = p.bias ? p.bias[c] : 0.0f;
    s1[i] = s2[i] = 0.0f;
  }
  const int64_t base = w.n * p.rows * p.C + w.col;
  Row<VEC> buf[4];
  if (w.here)
    rows_ahead(w, rpb, [&](int64_t r, Row<VEC>& v) {
      load_vec<T, VEC>((const T*)p.x + base + r * p.C, v.x);
      load_vec<T, VEC>((const T*)p.dy + base + r * p.C, v.dy);
      if (GATE) load_vec<T, VEC>((const T*)p.z + base + r * p.C, v.z);
    }, [&](int64_t, const Row<VEC>& v) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float dz;
        const float xh = (v.x[i] - mu[i]) * rs[i];
        const float du =
            Point<SILU, GATE>::backward(fmaf(xh, wt[i], sh[i]), GATE ? v.z[i] : 0.0f, v.dy[i], &dz);
        s1[i] += du;
        s2[i] = fmaf(du, xh, s2[i]);
      }
    }, buf);
  __shared__ float2 all[256];
  float2* const part = (float2*)p.ws + (int64_t)w.block * p.C;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    float2 t = make_float2(s1[i], s2[i]);
    if (rpb > 1) {
      __syncthreads();
      all[threadIdx.x] = t;
      __syncthreads();
      if (w.r0 == 0)
        for (int r = 1; r < rpb; ++r) {
          const float2 o = all[threadIdx.x + r * tile];
          t.x += o.x;
          t.y += o.y;
        }
    }
    if (w.here && w.r0 == 0) part[w.col + i] = t;
  }
}

// One block per (entry, group) and slice: sum dn / M and sum(dn xh) / M, M the
// whole group's.
__global__ __launch_bounds__(256) void merge_grads_kernel(const Args p, int slice_pieces, float2* out) {
  __shared__ float scratch[4];
  const Slice sl = slice_of(p, slice_pieces);
  if (sl.n >= p.batch) return;
  const int g = sl.g, cg = sl.cg;
  const float2* const part = sl.part;
  const int64_t m = sl.m;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < m; i += 256) {
    const int64_t piece = i / cg;
    const int c = (int)(i - piece * cg);
    const float2 e = part[piece * p.C + c];
    const float wt = p.weight ? p.weight[g * cg + c] : 1.0f;
    s1 = fmaf(wt, e.x, s1);
    s2 = fmaf(wt, e.y, s2);
  }
  const float inv = 1.0f / ((float)p.rows * (float)cg);
  s1 = block_sum(s1, scratch) * inv;
  s2 = block_sum(s2, scratch) * inv;
  if (threadIdx.x == 0) out[(int64_t)sl.group * gridDim.y + blockIdx.y] = make_float2(s1, s2);
}

__global__ __launch_bounds__(256) void join_grads_kernel(const float2* part, int slices, int64_t n, float2* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float2 a = part[i * slices];
  for (int k = 1; k < slices; ++k) {
    const float2 e = part[i * slices + k];
    a.x += e.x;
    a.y += e.y;
  }
  out[i] = a;
}

template <typename T, int VEC, bool SILU, bool GATE>
__global__ __launch_bounds__(256) void apply_bwd_kernel(const Args p, const float2* sums, int tile, int rpb) {
  const Where w = where<VEC>(p, tile, rpb);
  if (!w.here || w.n >= p.batch) return;
  const int cg = p.C / p.groups;
  float mu[VEC], rs[VEC], wt[VEC], sh[VEC], a1[VEC], a2[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = w.col + i;
    const int64_t at = w.n * p.groups + c / cg;
    mu[i] = p.mean[at];
    rs[i] = p.rstd[at];
    wt[i] = p.weight ? p.weight[c] : 1.0f;
    sh[i] = p.bias ? p.bias[c] : 0.0f;
    const float2 s = sums[at];
    a1[i] = s.x;
    a2[i] = s.y;
  }
  const int64_t base = w.n * p.rows * p.C + w.col;
  Row<VEC> buf[4];
  rows_ahead(w, rpb, [&](int64_t r, Row<VEC>& v) {
    load_vec<T, VEC>((const T*)p.x + base + r * p.C, v.x);
    load_vec<T, VEC>((const T*)p.dy + base + r * p.C, v.dy);
    if (GATE) load_vec<T, VEC>((const T*)p.z + base + r * p.C, v.z);
  }, [&](int64_t r, const Row<VEC>& v) {
    float dz[VEC], dx[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float xh = (v.x[i] - mu[i]) * rs[i];
      const float du =
          Point<SILU, GATE>::backward(fmaf(xh, wt[i], sh[i]), GATE ? v.z[i] : 0.0f, v.dy[i], &dz[i]);
      dx[i] = rs[i] * (du * wt[i] - a1[i] - xh * a2[i]);
    }
    store_vec<T, VEC>((T*)p.dx + base + r * p.C, dx);
    if (GATE) store_vec<T, VEC>((T*)p.dz + base + r * p.C, dz);
  }, buf);
}

// db and dw: `rows` rows of partial sums (db, dw per channel) added in a fixed
// order, 16 channels and 64 row groups per block.
__global__ __launch_bounds__(1024) void sum_channels_kernel(const float2* part, int64_t rows, int C,
                                                            float* dweight, float* dbias) {
  __shared__ float2 all[64][17];
  const int ch = threadIdx.x & 15, c = blockIdx.x * 16 + ch, rg = threadIdx.x >> 4;
  float s1 = 0.0f, s2 = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int64_t r = rg; r < rows; r += 64) {
      const float2 e = part[r * C + c];
      s1 += e.x;
      s2 += e.y;
    }
  }
  all[rg][ch] = make_float2(s1, s2);
  for (int half = 32; half > 0; half >>= 1) {
    __syncthreads();
    if (rg < half) {
      all[rg][ch].x += all[rg + half][ch].x;
      all[rg][ch].y += all[rg + half][ch].y;
    }
  }
  if (rg == 0 && c < C) {
    if (dbias) dbias[c] = all[0][ch].x;
    if (dweight) dweight[c] = all[0][ch].y;
  }
}

// ---- host ---------------------------------------------------------------------

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Plan {
  bool rows;            // the one-row form
  int vec, lpg, nv;     // one-row form: channels per vector, lanes per group, vectors per lane
  int tile, rpb, tiles; // slots (one-row) or vector columns of a block, rows at a time, blocks across
  int64_t blocks;       // one-row form: blocks down the entries
  int pieces;           // otherwise: pieces of an entry's rows
  int64_t piece_rows;
  int slices, slice_pieces;  // of a group's pieces, merged apart and joined
};

// channels of the widest access (at most `cap`) that the pointers and a run of
// `len` channels allow
int widest(const Args& p, bool f32, int64_t len, int cap) {
  const int most = cap < (f32 ? 4 : 8) ? cap : (f32 ? 4 : 8);
  const void* io[6] = {p.x, p.z, p.y, p.dy, p.dx, p.dz};
  int v = most;
  for (; v > 1; v /= 2) {
    bool ok = len % v == 0;
    for (const void* q : io) ok = ok && ((uintptr_t)q % (v * (f32 ? 4 : 2))) == 0;
    if (ok) break;
  }
  return v;
}

Plan plan(const Args& p, bool f32, bool bwd, int cap = 8) {
  Plan l = {};
  const int cg = p.C / p.groups;
  l.vec = widest(p, f32, cg, cap);
  const int vecs = cg / l.vec;
  l.lpg = 1;
  while (l.lpg < 64 && l.lpg < vecs) l.lpg *= 2;
  l.nv = 1;
  while (l.nv < 4 && l.lpg * l.nv < vecs) l.nv *= 2;
  l.rows = p.rows == 1 && l.lpg * l.nv >= vecs;
  if (l.rows) {
    const int64_t slots = (int64_t)p.groups * l.lpg;
    l.tile = (int)(slots < 256 ? slots : 256);
    l.tiles = (int)((slots + l.tile - 1) / l.tile);
    l.rpb = 256 / l.tile;
    const int64_t most = (p.batch + l.rpb - 1) / l.rpb;
    const int64_t want = ((bwd ? 1024 : 2048) + l.tiles - 1) / l.tiles;
    l.blocks = most < want ? most : want;
    return l;
  }
  l.vec = widest(p, f32, p.C, cap);
  const int cols = p.C / l.vec;
  l.tile = cols < 256 ? cols : 256;
  l.tiles = (cols + l.tile - 1) / l.tile;
  l.rpb = 256 / l.tile;
  // pieces: about 1024 blocks (four per CU), and at least 8 rows for each thread
  // of one, so that the partial sums (8 bytes per channel and piece) stay well
  // below the tensor's own bytes.  An entry of fewer rows is one piece all the
  // same: one row of a group too wide for the registers of a wave (over 2048 bf16
  // or 1024 fp32 channels, over 256 of an odd number) moves 22 bytes a bf16
  // channel forwards where 4 are needed.
  int64_t pieces = (1024 + p.batch * l.tiles - 1) / (p.batch * l.tiles);
  const int64_t most = (p.rows + 8 * l.rpb - 1) / (8 * l.rpb);
  if (pieces > most) pieces = most;
  if (pieces < 1) pieces = 1;
  l.piece_rows = (p.rows + pieces - 1) / pieces;
  if (l.piece_rows < 1) l.piece_rows = 1;
  l.pieces = (int)((p.rows + l.piece_rows - 1) / l.piece_rows);
  if (l.pieces < 1) l.pieces = 1;
  // Few wide groups leave their merge to a few blocks with much to read (32
  // groups of 256 channels, 256 pieces: 184 us forwards in one slice, 52 in
  // 16): about 4096 entries to a slice.  Below 8192 the second launch costs more.
  const int64_t entries = (int64_t)l.pieces * cg;
  int64_t slices = entries > 8192 ? (entries + 4095) / 4096 : 1;
  if (slices > 32) slices = 32;
  if (slices > l.pieces) slices = l.pieces;
  l.slice_pieces = (int)((l.pieces + slices - 1) / slices);
  l.slices = (int)((l.pieces + l.slice_pieces - 1) / l.slice_pieces);
  return l;
}

template <typename T, int VEC, int LPG, int NV>
hipError_t run_rows(const Args& p, const Plan& l, bool bwd, hipStream_t s) {
  const dim3 grid((uint32_t)l.blocks, (uint32_t)l.tiles);
  const int threads = (l.tile * l.rpb + 63) / 64 * 64;
#define SSM_GN(SILU, GATE)                                                                    \
  do {                                                                                        \
    if (bwd) rows_bwd_kernel<T, VEC, LPG, NV, SILU, GATE><<<grid, threads, 0, s>>>(p, l.tile, l.rpb); \
    else rows_fwd_kernel<T, VEC, LPG, NV, SILU, GATE><<<grid, threads, 0, s>>>(p, l.tile, l.rpb);     \
  } while (0)
  if (p.silu && p.z) SSM_GN(true, true);
  else if (p.silu) SSM_GN(true, false);
  else if (p.z) SSM_GN(false, true);
  else SSM_GN(false, false);
#undef SSM_GN
  return hipGetLastError();
}

template <typename T, int VEC, int LPG>
hipError_t run_rows_nv(const Args& p, const Plan& l, bool bwd, hipStream_t s) {
  if constexpr (LPG == 64) {
    if (l.nv == 4) return run_rows<T, VEC, LPG, 4>(p, l, bwd, s);
    if (l.nv == 2) return run_rows<T, VEC, LPG, 2>(p, l, bwd, s);
  }
  return run_rows<T, VEC, LPG, 1>(p, l, bwd, s);
}

template <typename T, int VEC>
hipError_t run_rows_lpg(const Args& p, const Plan& l, bool bwd, hipStream_t s) {
  switch (l.lpg) {
    case 1: return run_rows_nv<T, VEC, 1>(p, l, bwd, s);
    case 2: return run_rows_nv<T, VEC, 2>(p, l, bwd, s);
    case 4: return run_rows_nv<T, VEC, 4>(p, l, bwd, s);
    case 8: return run_rows_nv<T, VEC, 8>(p, l, bwd, s);
    case 16: return run_rows_nv<T, VEC, 16>(p, l, bwd, s);
    case 32: return run_rows_nv<T, VEC, 32>(p, l, bwd, s);
    default: return run_rows_nv<T, VEC, 64>(p, l, bwd, s);
  }
}

// the parts of a workspace: partial sums, the groups' two numbers, the slices'
size_t parts_bytes(const Args& p, const Plan& l, bool bwd) {
  if (l.rows) return bwd ? up256((size_t)l.blocks * p.C * 8) : 0;
  return up256((size_t)p.batch * l.pieces * p.C * 8);
}

template <typename T, int VEC, bool SILU, bool GATE>
hipError_t run_pieces(const Args& q, const Plan& l, bool bwd, hipStream_t s) {
  Args p = q;
  p.pieces = l.pieces;
  p.piece_rows = l.piece_rows;
  const int threads = (l.tile * l.rpb + 63) / 64 * 64;
  const int64_t ng = p.batch * p.groups;
  const Grid gp = grid_of(p.batch * l.pieces, threads), gg = grid_of(ng, 256);
  const dim3 grid(gp.x, (uint32_t)l.tiles, gp.more);
  const dim3 groups(gg.x, (uint32_t)l.slices, gg.more), join((uint32_t)((ng + 255) / 256));
  char* const extra = (char*)p.ws + parts_bytes(p, l, bwd);
  void* const slices = extra + up256((size_t)ng * 8);
  hipError_t e;
  if (!bwd) {
    piece_stats_kernel<T, VEC><<<grid, threads, 0, s>>>(p, l.tile, l.rpb);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    float* const mean = p.mean ? p.mean : (float*)extra;
    float* const rstd = p.rstd ? p.rstd : (float*)extra + (size_t)p.batch * p.groups;
    merge_stats_kernel<<<groups, 256, 0, s>>>(p, l.slice_pieces, (float4*)slices, mean, rstd);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (l.slices > 1) {
      join_stats_kernel<<<join, 256, 0, s>>>((const float4*)slices, l.slices, ng, p.eps, mean, rstd);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    apply_fwd_kernel<T, VEC, SILU, GATE><<<grid, threads, 0, s>>>(p, mean, rstd, l.tile, l.rpb);
    return hipGetLastError();
  }
  piece_grads_kernel<T, VEC, SILU, GATE><<<grid, threads, 0, s>>>(p, l.tile, l.rpb);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  merge_grads_kernel<<<groups, 256, 0, s>>>(p, l.slice_pieces, (float2*)(l.slices > 1 ? slices : extra));
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (l.slices > 1) {
    join_grads_kernel<<<join, 256, 0, s>>>((const float2*)slices, l.slices, ng, (float2*)extra);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  apply_bwd_kernel<T, VEC, SILU, GATE><<<grid, threads, 0, s>>>(p, (const float2*)extra, l.tile, l.rpb);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t run_pieces_act(const Args& p, const Plan& l, bool bwd, hipStream_t s) {
  if (p.silu && p.z) return run_pieces<T, VEC, true, true>(p, l, bwd, s);
  if (p.silu) return run_pieces<T, VEC, true, false>(p, l, bwd, s);
  if (p.z) return run_pieces<T, VEC, false, true>(p, l, bwd, s);
  return run_pieces<T, VEC, false, false>(p, l, bwd, s);
}

template <typename T>
hipError_t run(const Args& p, const Plan& l, bool bwd, hipStream_t s) {
  constexpr int kMost = sizeof(T) == 4 ? 4 : 8;
  if (l.vec == kMost) return l.rows ? run_rows_lpg<T, kMost>(p, l, bwd, s) : run_pieces_act<T, kMost>(p, l, bwd, s);
  if (l.vec == 4) return l.rows ? run_rows_lpg<T, 4>(p, l, bwd, s) : run_pieces_act<T, 4>(p, l, bwd, s);
  if (l.vec == 2) return l.rows ? run_rows_lpg<T, 2>(p, l, bwd, s) : run_pieces_act<T, 2>(p, l, bwd, s);
  return l.rows ? run_rows_lpg<T, 1>(p, l, bwd, s) : run_pieces_act<T, 1>(p, l, bwd, s);
}

size_t total_bytes(const Args& p, const Plan& l, bool bwd) {
  return parts_bytes(p, l, bwd) + (l.rows ? 0
                                               : up256((size_t)p.batch * p.groups * 8) +
                                                     (l.slices > 1 ? up256((size_t)p.batch * p.groups * l.slices * 16)
                                                                   : 0));
}

}  // namespace

bool fits(const Args& p, bool f32, bool bwd) {
  if (p.batch == 0 || p.rows == 0) return true;
  if (p.batch > 0x7fffffff / p.groups) return false;
  for (int cap = 8; cap >= 1; cap /= 2) {
    const Plan l = plan(p, f32, bwd, cap);
    if (l.tiles > 65535 || (!l.rows && p.batch > 0x7fffffff / l.pieces)) return false;
  }
  return true;
}

size_t workspace_bytes(const Args& p, bool f32, bool bwd) {
  if (p.batch == 0 || p.rows == 0) return 0;
  Args q = p;
  q.x = q.z = q.dy = nullptr;
  q.y = q.dx = q.dz = nullptr;
  size_t need = 0;
  for (int cap = 8; cap >= 1; cap /= 2) {
    const size_t n = total_bytes(q, plan(q, f32, bwd, cap), bwd);
    need = n > need ? n : need;
  }
  return need;
}

hipError_t forward(const Args& p, bool f32, hipStream_t s) {
  if (p.batch == 0 || p.rows == 0) return hipSuccess;
  const Plan l = plan(p, f32, false);
  return f32 ? run<float>(p, l, false, s) : run<bf16_bits>(p, l, false, s);
}

hipError_t backward(const Args& p, bool f32, hipStream_t s) {
  int64_t rows = 0;
  if (p.batch > 0 && p.rows > 0) {
    const Plan l = plan(p, f32, true);
    const hipError_t e = f32 ? run<float>(p, l, true, s) : run<bf16_bits>(p, l, true, s);
    if (e != hipSuccess) return e;
    rows = l.rows ? l.blocks : p.batch * l.pieces;
  }
  if (p.dweight || p.dbias) {
    sum_channels_kernel<<<dim3((uint32_t)((p.C + 15) / 16)), 1024, 0, s>>>((const float2*)p.ws, rows, p.C,
                                                                          p.dweight, p.dbias);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace group_norm
}  // namespace ssm66
