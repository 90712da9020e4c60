// rotary.hip -- rotary positions of queries and keys.
//
// Pair j of a head is turned by the angle t = position * freqs[j]:
//   (a, b) -> mscale (a cos t - b sin t, b cos t + a sin t),
// a and b the elements 2j and 2j + 1 (interleaved) or j and j + pairs (halves).
// The gradient is the turn by -t.
//
// HBM bounds it: 8 x 2048 tokens, 24 + 8 heads of 128, half of each turned, bf16,
// 51 us (268 MB, a copy's rate; a head at a time and up to 32 heads a thread, 67).
// A thread keeps the cosines and sines of its pairs of one token and goes over the
// heads of queries and keys with them, 16 bytes an access (the two halves of a pair
// are two); few tokens are spread over the heads too.  A thread's heads are one in
// so many, so that threads beside each other have heads beside each other:
// 8 x 2048 tokens, 16 + 16 heads of 40, 20 turned as halves, bf16, 31 us a turn
// (heads in a row, 36; and 4 bytes an access in the copied part, 41; 2 bytes, 50);
// heads of 128 as halves lose 1%.
//
// Angles: position * freqs / 2 pi in fp64 (2^31 positions leave 6e-8 of a turn),
// less the nearest quarter turn, then the series of sine and cosine up to an
// eighth of a turn in fp32, which leave out less than 2e-9.
#include "lm_grid.h"
#include "rotary_launch.h"
#include "vec_io.h"

namespace ssm66 {
namespace rotary {

namespace {

__device__ __forceinline__ void turn_of(int position, float freq, float* c, float* s) {
  const double rev = (double)position * (double)freq * 0.15915494309189535;
  const double quarter = rint(rev * 4.0);
  const float x = (float)((rev - quarter * 0.25) * 6.283185307179586);
  const int k = (int)((int64_t)quarter & 3);
  const float z = x * x;
  float sn = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(z, sn, 8.3333333e-3f);
  sn = fmaf(z, sn, -1.6666667e-1f);
  sn = fmaf(x * z, sn, x);
  float cs = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(z, cs, -1.3888889e-3f);
  cs = fmaf(z, cs, 4.1666667e-2f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.0f);
  const float a = k & 1 ? sn : cs, b = k & 1 ? cs : sn;
  *c = k == 1 || k == 2 ? -a : a;
  *s = k >= 2 ? -b : b;
}

// BYTES of memory as they are, from any address of a value
template <int BYTES> struct Piece {
  typedef uint32_t type __attribute__((ext_vector_type(BYTES / 4), aligned(2)));
};
template <> struct Piece<4> { typedef uint32_t type __attribute__((aligned(2))); };
template <> struct Piece<2> { typedef uint16_t type; };
// N elements of each of a thread's heads
template <typename T, int N>
__device__ __forceinline__ void copy(const Args& p, const T* q, const T* k, T* qo, T* ko, int split) {
  typedef typename Piece<N * sizeof(T)>::type P;
  const int heads = p.H + p.Hk;
  for (int g0 = split; g0 < heads; g0 += 4 * p.splits) {
    P v[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int h = g0 + g * p.splits;
      if (h < heads) v[g] = *(const P*)((h < p.H ? q : k) + (int64_t)(h < p.H ? h : h - p.H) * p.D);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int h = g0 + g * p.splits;
      if (h < heads) *(P*)((h < p.H ? qo : ko) + (int64_t)(h < p.H ? h : h - p.H) * p.D) = v[g];
    }
  }
}

// VEC elements an access.  Interleaved: a thread has one access, VEC / 2 pairs
// (VEC == 1: one pair as two elements).  Halves: two accesses, VEC pairs.  The
// threads past the pairs copy what is not turned.  N: unsigned of 32 bits where
// the number of threads fits (a 64-bit quotient costs as much as four heads).
template <typename T, int VEC, bool INTER, typename N>
__global__ __launch_bounds__(256) void rotary_kernel(const Args p) {
  constexpr int W = INTER ? (VEC == 1 ? 2 : VEC) : VEC;      // elements from one thread to the next
  constexpr int PAIRS = INTER ? W / 2 : VEC;
  constexpr int kAhead = INTER ? 4 : 2;  // heads loaded before the first is stored
  const N n = ((N)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
  const N rest = n / (N)p.lanes;
  const int lane = (int)(n - rest * (N)p.lanes);
  const int64_t tok = (int64_t)(rest / (N)p.splits);
  const int split = (int)(rest - (N)tok * (N)p.splits);
  if (tok >= p.tokens) return;
  const int turning = INTER ? 2 * p.pairs / W : p.pairs / VEC;
  const int heads = p.H + p.Hk, step = p.splits;
  const bool turns = lane < turning;
  // copied: 16 bytes an access wherever there are as many, the last one overlapping
  // the one before it (both store the same)
  constexpr int FULL = 16 / sizeof(T);
  const int copied = p.D - 2 * p.pairs, piece = lane - turning;
  int col = lane * W;
  if (!turns) col = 2 * p.pairs + (copied >= FULL ? min(piece * FULL, copied - FULL) : piece * VEC);
  const T* const q = (const T*)p.q + tok * p.H * p.D + col;
  const T* const k = (const T*)p.k + tok * p.Hk * p.D + col;
  T* const qo = (T*)p.qo + tok * p.H * p.D + col;
  T* const ko = (T*)p.ko + tok * p.Hk * p.D + col;
  if (!turns) {
    if (copied >= FULL) copy<T, FULL>(p, q, k, qo, ko, split);
    else copy<T, VEC>(p, q, k, qo, ko, split);
    return;
  }
  const int position = p.positions ? p.positions[tok] : (int)((N)tok % (N)p.L);
  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int j = 0; j < PAIRS; ++j) {
    turn_of(position, p.freqs[lane * PAIRS + j], &c[j], &s[j]);
    c[j] *= p.mscale;
    s[j] *= p.mscale * p.sign;
  }
  for (int g0 = split; g0 < heads; g0 += kAhead * step) {
    float a[kAhead][W], b[INTER ? 1 : kAhead][VEC];
#pragma unroll
    for (int g = 0; g < kAhead; ++g) {
      const int h = g0 + g * step;
      if (h >= heads) break;
      const T* const in = (h < p.H ? q : k) + (int64_t)(h < p.H ? h : h - p.H) * p.D;
      load_n<W>(in, a[g]);
      if constexpr (!INTER) load_n<VEC>(in + p.pairs, b[g]);
    }
#pragma unroll
    for (int g = 0; g < kAhead; ++g) {
      const int h = g0 + g * step;
      if (h >= heads) break;
      T* const out = (h < p.H ? qo : ko) + (int64_t)(h < p.H ? h : h - p.H) * p.D;
      if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          const float x = a[g][2 * j], y = a[g][2 * j + 1];
          a[g][2 * j] = fmaf(x, c[j], -(y * s[j]));
          a[g][2 * j + 1] = fmaf(y, c[j], x * s[j]);
        }
        store_n<W>(out, a[g]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float x = a[g][j], y = b[g][j];
          a[g][j] = fmaf(x, c[j], -(y * s[j]));
          b[g][j] = fmaf(y, c[j], x * s[j]);
        }
        store_n<VEC>(out, a[g]);
        store_n<VEC>(out + p.pairs, b[g]);
      }
    }
  }
}

template <typename T, int VEC, bool INTER>
hipError_t launch(Args p, hipStream_t s) {
  constexpr int W = INTER ? (VEC == 1 ? 2 : VEC) : VEC;
  const bool in_place = p.q == p.qo && p.k == p.ko;
  constexpr int FULL = 16 / sizeof(T);
  const int copied = p.D - 2 * p.pairs;
  p.lanes = INTER ? 2 * p.pairs / W : p.pairs / VEC;
  if (!in_place) p.lanes += copied >= FULL ? (copied + FULL - 1) / FULL : copied / VEC;
  // a thread takes up to eight heads (the angles cost as much as three), fewer
  // where that leaves less than eight waves a CU
  const int heads = p.H + p.Hk;
  const int64_t wide = p.tokens * p.lanes, want = 256 * 8 * 64;
  int64_t splits = (want + wide - 1) / wide;
  if (splits < (heads + 7) / 8) splits = (heads + 7) / 8;
  if (splits > heads) splits = heads;
  const int each = (int)((heads + splits - 1) / splits);
  p.splits = (heads + each - 1) / each;
  const int64_t n = wide * p.splits;
  const Grid g = grid_of((n + 255) / 256, 256);
  const dim3 grid(g.x, g.more);
  if (n < 0xffff0000ll) rotary_kernel<T, VEC, INTER, uint32_t><<<grid, 256, 0, s>>>(p);
  else rotary_kernel<T, VEC, INTER, uint64_t><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t layouts(const Args& p, hipStream_t s) {
  return p.interleaved ? launch<T, VEC, true>(p, s) : launch<T, VEC, false>(p, s);
}

template <typename T>
hipError_t pick(const Args& p, hipStream_t s) {
  // 16 bytes an access where the turned and the copied part of a head are whole
  // multiples of them, else 8, 4 of bf16, a value
  constexpr int VEC = 16 / sizeof(T);
  const int parts = p.D | (p.interleaved ? 2 * p.pairs : p.pairs);  // divided by a power of two if both are
  if (parts % VEC == 0) return layouts<T, VEC>(p, s);
  if (parts % (VEC / 2) == 0) return layouts<T, VEC / 2>(p, s);
  if (VEC == 8 && parts % 2 == 0) return layouts<T, VEC / 4>(p, s);
  return layouts<T, 1>(p, s);
}

}  // namespace

bool fits(int64_t tokens, int heads, int D) {
  // one thread an element at most, 32-bit block numbers
  return (__int128)tokens * heads * D < (__int128)1 << 38;
}

hipError_t run(const Args& p, bool f32, hipStream_t s) {
  return f32 ? pick<float>(p, s) : pick<bf16_bits>(p, s);
}

}  // namespace rotary
}  // namespace ssm66
