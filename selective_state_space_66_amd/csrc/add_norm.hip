// add_norm.hip -- a residual, a dropped-out branch, and the norm of their sum.
//
//   h = residual + dropout(x),  in h's type,
//   layer: xh = (h - mean) rstd, rstd = 1 / sqrt(sum (h - mean)^2 / n + eps);
//   RMS:   xh = h rstd,          rstd = 1 / sqrt(sum h^2 / n + eps);
//   y = xh w + b.
// Backwards, with dn = dy w and dh what reaches h from elsewhere,
//   dH = rstd (dn - [sum dn / n] - xh sum(dn xh) / n) + dh   ([]: layer only),
//   dresidual = dH,  dx = dropout's map of dH,  dw = sum dy xh,  db = sum dy.
//
// HBM bounds all of it: 16384 x 1536, bf16 with an fp32 stream and dropout,
// forwards 59 us (302 MB, at a copy's 5.1 TB/s; 65 in a training step, behind a
// backward call), backwards 80 (403 MB, 5.0) and 5 for the column sums.  A row is
// read once and held by 16 to 64 lanes or by two to sixteen waves, eight
// neighbouring values a lane (sixteen past 8192); the sums go over the lanes by
// shuffles and over the waves through LDS.  A thread keeps its columns over all the
// rows it takes, so the backward adds dw and db in registers; a block leaves one
// row of partial sums, added up in a fixed order by a kernel of its own.  All sums
// are fp32, those over the rows' blocks fp64.
#include "add_norm_launch.h"
#include "vec_io.h"

namespace ssm66 {
namespace add_norm {

namespace {

constexpr int VEC = 8;

constexpr int threads_of(int lanes) { return lanes > 128 ? lanes : 256; }
// LPR lanes hold a row, VECS times eight neighbouring values each.
template <int LPR>
struct Form {
  static constexpr int kThreads = threads_of(LPR);
  static constexpr int kRows = kThreads / LPR;  // of a block at a time
};

// how many of the eight values from column c on the row has (EVEN: rows are
// multiples of eight, all or none)
template <bool EVEN>
__device__ __forceinline__ int values_at(int c, int dim) {
  return c < dim ? (EVEN || dim - c >= VEC ? VEC : dim - c) : 0;
}
template <bool EVEN, typename T>
__device__ __forceinline__ void load(Raw8<T>& r, const T* p, int n) {
  if constexpr (EVEN) {
    if (n > 0) r.load(p, VEC);
    else r = Raw8<T>{};
  } else {
    r.load(p, n);
  }
}

// The factors of eight values of a row; rows of a multiple of four begin at one.
template <bool EVEN>
__device__ __forceinline__ void factors(const Args& p, uint64_t seed, uint64_t offset, int64_t at,
                                        float (&f)[VEC]) {
  if (EVEN || p.dim % 4 == 0) drop_factors(p.drop, seed, offset, at, f);
  else drop_factors_any(p.drop, seed, offset, at, f);
}

// Sums of two values over the lanes of a row, to all of them.  `part` has room
// for the waves of a block; a second call uses the other half.
template <int LPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float2* part) {
#pragma unroll
  for (int m = (LPR < 64 ? LPR : 64) / 2; m > 0; m >>= 1) {
    a += __shfl_xor(a, m);
    b += __shfl_xor(b, m);
  }
  if constexpr (LPR > 64) {
    constexpr int N = LPR / 64;
    const int w = (int)threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[w] = make_float2(a, b);
    __syncthreads();
    const float2* const mine = part + w / N * N;
    a = b = 0.0f;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      a += mine[q].x;
      b += mine[q].y;
    }
  }
}

template <typename T, typename TH, int LPR, int VECS, bool EVEN>
__global__ __launch_bounds__(Form<LPR>::kThreads) void fwd_kernel(const Args p) {
  typedef Form<LPR> F;
  __shared__ float2 part[2][16];
  const int l = (int)threadIdx.x % LPR;
  const int64_t r0 = (int64_t)blockIdx.x * F::kRows + (int)threadIdx.x / LPR;
  const int64_t step = (int64_t)gridDim.x * F::kRows;
  const float inv = 1.0f / (float)p.dim;
  uint64_t seed = 0, offset = 0;
  if (p.drop.rng) {
    seed = (uint64_t)p.drop.rng[0];
    offset = (uint64_t)p.drop.rng[1] + p.drop.site;
  }
  float w[VECS][VEC], b[VECS][VEC];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int c = (l + j * LPR) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      w[j][k] = p.weight && c + k < p.dim ? p.weight[c + k] : 1.0f;
      b[j][k] = p.bias && c + k < p.dim ? p.bias[c + k] : 0.0f;
    }
  }
  // whole blocks stay for the barriers: the rows past the last are empty.  A row
  // is on its way while the one before it is worked on.
  const int64_t rounds = (p.rows + step - 1) / step;
  Raw8<T> nx[VECS];
  Raw8<TH> nr[VECS];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = (l + j * LPR) * VEC, n = row < p.rows ? values_at<EVEN>(c, p.dim) : 0;
      load<EVEN>(nx[j], (const T*)p.x + row * p.dim + c, n);
      load<EVEN>(nr[j], (const TH*)p.residual + row * p.dim + c, p.residual ? n : 0);
    }
  };
  fetch(r0);
  for (int64_t q = 0; q < rounds; ++q) {
    const int64_t row = r0 + q * step;
    const bool real = row < p.rows;
    const int64_t base = row * p.dim;
    float v[VECS][VEC], res[VECS][VEC];
    float s = 0.0f, sq = 0.0f;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      nx[j].get(v[j]);
      nr[j].get(res[j]);
    }
    fetch(row + step);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = (l + j * LPR) * VEC;
      if (real && c < p.dim) {  // (elsewhere, and past the row's end, all is zero)
        if (p.drop.rng) {
          float f[VEC];
          factors<EVEN>(p, seed, offset, base + c, f);
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[j][k] = dropped(v[j][k], f[k]);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[j][k] = as_stored(v[j][k] + res[j][k], (const TH*)nullptr);
        if (p.h) store_8((TH*)p.h + base + c, v[j], values_at<EVEN>(c, p.dim));
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        s += v[j][k];
        sq = fmaf(v[j][k], v[j][k], sq);
      }
    }
    row_sums<LPR>(s, sq, part[0]);
    float mean = 0.0f, var = sq * inv;
    if (!p.rms) {
      // the squares about the mean as rounded, and what the rounding left of it
      mean = s * inv;
      float left = 0.0f;
      sq = 0.0f;
#pragma unroll
      for (int j = 0; j < VECS; ++j) {
        const int n = values_at<EVEN>((l + j * LPR) * VEC, p.dim);
        const bool in = n > 0;
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[j][k] = in ? v[j][k] - mean : 0.0f;
        if (!EVEN)
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[j][k] = k < n ? v[j][k] : 0.0f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          left += v[j][k];
          sq = fmaf(v[j][k], v[j][k], sq);
        }
      }
      row_sums<LPR>(left, sq, part[1]);
      left *= inv;
      var = fmaf(-left, left, sq * inv);
      var = var < 0.0f ? 0.0f : var;  // (a NaN stays one)
      mean += left;
#pragma unroll
      for (int j = 0; j < VECS; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[j][k] -= left;
    }
    const float rstd = 1.0f / sqrtf(var + p.eps);
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = (l + j * LPR) * VEC;
      if (real && c < p.dim) {
        float y[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] = fmaf(v[j][k] * rstd, w[j][k], b[j][k]);
        store_8((T*)p.y + base + c, y, values_at<EVEN>(c, p.dim));
      }
    }
    if (real && l == 0) {
      if (p.mean && !p.rms) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    if constexpr (LPR > 64) __syncthreads();  // part[0] has been read
  }
}

template <typename T, typename TH, int LPR, int VECS, bool EVEN>
__global__ __launch_bounds__(Form<LPR>::kThreads) void bwd_kernel(const Args p) {
  typedef Form<LPR> F;
  __shared__ float2 part[2][16];
  const int l = (int)threadIdx.x % LPR;
  const int64_t r0 = (int64_t)blockIdx.x * F::kRows + (int)threadIdx.x / LPR;
  const int64_t step = (int64_t)gridDim.x * F::kRows;
  const float inv = 1.0f / (float)p.dim;
  uint64_t seed = 0, offset = 0;
  if (p.drop.rng) {
    seed = (uint64_t)p.drop.rng[0];
    offset = (uint64_t)p.drop.rng[1] + p.drop.site;
  }
  float w[VECS][VEC], dw[VECS][VEC], db[VECS][VEC];
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    const int c = (l + j * LPR) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      w[j][k] = p.weight && c + k < p.dim ? p.weight[c + k] : 1.0f;
      dw[j][k] = db[j][k] = 0.0f;
    }
  }
  const int64_t rounds = (p.rows + step - 1) / step;
  for (int64_t q = 0; q < rounds; ++q) {
    const int64_t row = r0 + q * step;
    const bool real = row < p.rows;
    const int64_t base = row * p.dim;
    constexpr bool kLate = VECS > 1;  // dh loaded where it is needed: registers
    float xh[VECS][VEC], dy[VECS][VEC];
    Raw8<TH> rh[VECS];
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = (l + j * LPR) * VEC, n = real ? values_at<EVEN>(c, p.dim) : 0;
      Raw8<TH> a;
      Raw8<T> b;
      load<EVEN>(a, (const TH*)p.h + base + c, n);
      load<EVEN>(b, (const T*)p.dy + base + c, n);
      if (!kLate) load<EVEN>(rh[j], (const TH*)p.dh + base + c, p.dh ? n : 0);
      a.get(xh[j]);
      b.get(dy[j]);
    }
    const float mean = real && !p.rms ? p.mean[row] : 0.0f, rstd = real ? p.rstd[row] : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < VECS; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        xh[j][k] = (xh[j][k] - mean) * rstd;  // past the row's end dy is 0
        dw[j][k] = fmaf(dy[j][k], xh[j][k], dw[j][k]);
        db[j][k] += dy[j][k];
        dy[j][k] *= w[j][k];
        s1 += dy[j][k];
        s2 = fmaf(dy[j][k], xh[j][k], s2);
      }
    row_sums<LPR>(s1, s2, part[q & 1]);
    s1 = p.rms ? 0.0f : s1 * inv;
    s2 *= inv;
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      const int c = (l + j * LPR) * VEC;
      if (real && c < p.dim) {
        const int n = values_at<EVEN>(c, p.dim);
        float g[VEC], dh[VEC];
        if (kLate) load<EVEN>(rh[j], (const TH*)p.dh + base + c, p.dh ? n : 0);
        rh[j].get(dh);
#pragma unroll
        for (int k = 0; k < VEC; ++k) g[k] = rstd * (dy[j][k] - s1 - xh[j][k] * s2) + dh[k];
        if (p.dresidual) store_8((TH*)p.dresidual + base + c, g, n);
        if (p.drop.rng) {
          float f[VEC];
          factors<EVEN>(p, seed, offset, base + c, f);
#pragma unroll
          for (int k = 0; k < VEC; ++k) g[k] = dropped(g[k], f[k]);
        }
        store_8((T*)p.dx + base + c, g, n);
      }
    }
  }
  if (!p.part) return;
  // the block's rows added in order, then one row of partial sums (dw, db)
  __shared__ float2 sums[F::kThreads];
#pragma unroll
  for (int j = 0; j < VECS; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int c = (l + j * LPR) * VEC + k;
      float2 t = make_float2(dw[j][k], db[j][k]);
      if (F::kRows > 1) {
        __syncthreads();
        sums[threadIdx.x] = t;
        __syncthreads();
        if ((int)threadIdx.x < LPR)
          for (int r = 1; r < F::kRows; ++r) {
            t.x += sums[threadIdx.x + r * LPR].x;
            t.y += sums[threadIdx.x + r * LPR].y;
          }
      }
      if ((int)threadIdx.x < LPR && c < p.dim) p.part[(int64_t)blockIdx.x * p.dim + c] = t;
    }
}

// dw and db from the blocks' partial sums: 16 columns of a block, 64 groups of
// lanes that take every 64th row, added in fp64 in a fixed order
__global__ __launch_bounds__(1024) void column_sum_kernel(const float2* part, float* dw, float* db,
                                                          int blocks, int dim) {
  constexpr int kGroups = 64;
  __shared__ double2 sums[kGroups][16];
  const int l = (int)threadIdx.x & 15, g = (int)threadIdx.x >> 4;
  const int c = (int)blockIdx.x * 16 + l;
  double x = 0.0, y = 0.0;
  if (c < dim) {
    int r = g;
    for (; r + 7 * kGroups < blocks; r += 8 * kGroups) {
      float2 t[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) t[q] = part[(int64_t)(r + kGroups * q) * dim + c];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x += t[q].x;
        y += t[q].y;
      }
    }
    for (; r < blocks; r += kGroups) {
      const float2 t = part[(int64_t)r * dim + c];
      x += t.x;
      y += t.y;
    }
  }
  for (int many = kGroups; many > 1; many /= 8) {  // 64, then 8 of them left
    sums[g][l] = make_double2(x, y);
    __syncthreads();
    if (g < many / 8) {
      for (int q = 1; q < 8; ++q) {
        const double2 t = sums[g + q * (many / 8)][l];
        x += t.x;
        y += t.y;
      }
    }
    __syncthreads();
  }
  if (g == 0 && c < dim) {
    if (dw) dw[c] = (float)x;
    if (db) db[c] = (float)y;
  }
}

// Blocks: as many as run at a time (256 CUs of about 1024 threads), so that each
// has its share of the rows at once (8192 x 4096, bf16 with fp32 h: forwards 83 us;
// 1.5 times as many blocks 94, a block a row 157).  Those of the backward each
// leave a row of partial sums; four of 192 threads take 87 us for 16384 x 1536,
// five 89.
constexpr int64_t most_blocks(int threads) { return 256 * (1024 / threads); }
constexpr int64_t back_most(int threads) { return 256 * (threads > 256 ? 1024 / threads : 4); }

// Lanes of a row, eight values each: the next power of two, and three waves; past
// 8192 each holds twice eight values.  Forwards and backwards, bf16 with fp32 h and
// dropout, three waves and four: 16384 x 1536 59 + 85 us, 64 + 86; 1280: 50 + 72, 55 +
// 73; 1032: 47 + 58, 52 + 58.  Five or ten waves are forwards faster alone, five
// slower backwards: 8192 x 2560 50 + 79, with 512 lanes 61 + 72; 4096 x 5120 62 + 73,
// with 1024 lanes 72 + 72.
constexpr int lanes_of(int64_t dim) {
  return dim <= 128 ? 16 : dim <= 256 ? 32 : dim <= 512 ? 64 : dim <= 1024 ? 128 : dim <= 1536 ? 192
       : dim <= 2048 ? 256 : dim <= 4096 ? 512 : 1024;
}
// The blocks of a launch, which the backward's workspace is sized by too.
constexpr int64_t blocks_of(int64_t rows, int lanes, bool back) {
  const int threads = threads_of(lanes), at_once = threads / lanes;
  const int64_t n = rows / at_once + (rows % at_once != 0), most = back ? back_most(threads) : most_blocks(threads);
  return n < most ? n : most;
}

struct Call {
  Args p;
  bool back;
  hipStream_t s;
};

template <typename T, typename TH, int LPR, int VECS, bool EVEN>
hipError_t launch(const Call& c) {
  const unsigned n = (unsigned)blocks_of(c.p.rows, LPR, c.back);
  if (c.back) bwd_kernel<T, TH, LPR, VECS, EVEN><<<n, threads_of(LPR), 0, c.s>>>(c.p);
  else fwd_kernel<T, TH, LPR, VECS, EVEN><<<n, threads_of(LPR), 0, c.s>>>(c.p);
  return hipGetLastError();
}

template <typename T, typename TH, bool EVEN>
hipError_t pick(const Call& c) {
  switch (lanes_of(c.p.dim)) {
    case 16: return launch<T, TH, 16, 1, EVEN>(c);
    case 32: return launch<T, TH, 32, 1, EVEN>(c);
    case 64: return launch<T, TH, 64, 1, EVEN>(c);
    case 128: return launch<T, TH, 128, 1, EVEN>(c);
    case 192: return launch<T, TH, 192, 1, EVEN>(c);
    case 256: return launch<T, TH, 256, 1, EVEN>(c);
    case 512: return launch<T, TH, 512, 1, EVEN>(c);
    default: return c.p.dim <= 8192 ? launch<T, TH, 1024, 1, EVEN>(c) : launch<T, TH, 1024, 2, EVEN>(c);
  }
}
// Rows that are no multiple of eight pay for the piece at their end (16384 x
// 1536: 65 and 86 us, by the kernels for any row 77 and 89).
template <typename T, typename TH>
hipError_t pick(const Call& c) {
  return c.p.dim % VEC == 0 ? pick<T, TH, true>(c) : pick<T, TH, false>(c);
}

hipError_t run(const Call& c, bool x_f32, bool h_f32) {
  if (x_f32) return pick<float, float>(c);
  return h_f32 ? pick<bf16_bits, float>(c) : pick<bf16_bits, bf16_bits>(c);
}

}  // namespace

size_t workspace_bytes(int64_t rows, int64_t dim) {
  return (size_t)((blocks_of(rows, lanes_of(dim), true) * dim * 8 + 255) / 256 * 256);
}

hipError_t forward(const Args& p, bool x_f32, bool h_f32, hipStream_t s) {
  return run(Call{p, false, s}, x_f32, h_f32);
}

hipError_t backward(const Args& p, bool x_f32, bool h_f32, hipStream_t s) {
  if (p.rows > 0) {
    const hipError_t e = run(Call{p, true, s}, x_f32, h_f32);
    if (e != hipSuccess) return e;
  }
  if (!p.dweight && !p.dbias) return hipSuccess;
  const int blocks = (int)blocks_of(p.rows, lanes_of(p.dim), true);
  column_sum_kernel<<<(p.dim + 15) / 16, 1024, 0, s>>>(p.part, p.dweight, p.dbias, blocks, p.dim);
  return hipGetLastError();
}

}  // namespace add_norm
}  // namespace ssm66
