// gated_scan.hip -- the gated linear recurrence: forward, gradients, one token.
//
//   v_t = decay_c sigmoid(r_t),  a_t = exp(-v_t),  m_t = sqrt(1 - a_t^2),
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t,   y_t = h_t.
// Backwards, with lam_t the gradient of h_t,
//   lam_t = dy_t + a_{t+1} lam_{t+1},
//   dx_t = lam_t m_t g_t,   di_t = lam_t m_t x_t g_t (1 - g_t),   g = sigmoid(i),
//   P_t = v_t dL/dv_t = lam_t (g_t x_t a_t^2 v_t / m_t - a_t v_t h_{t-1}),
//   dr_t = P_t (1 - sigmoid(r_t)),   ddecay = sum P_t / decay.
//
// One pass over the tensors.  A block takes 128 tokens of a tile of channels, a
// wave's row of 256 bytes wide; a wave takes 8 or 16 of the tokens, a thread
// one or two channels of them in registers, so that the recurrence itself is a
// chain of multiply-adds.  What a stretch of tokens does to a state is the pair
// (V, H): h -> exp(-V) h + H, V the sum of its v.  Pairs are joined over the
// waves in LDS and over the chunks through memory: a block publishes the pair
// of its chunk as one 64-bit word, waits for the words of the chunks before it
// in its group of 32 chunks and for the state before the group, and goes on
// with its tokens, which never left the registers.  The order of every join is
// fixed by the chunk's number, so repeated calls give identical bits.
//
// Why the waits end: a block takes its chunk's number from a counter, chunks of
// every row in order, and waits only for words of smaller numbers.  The block
// with the smallest unfinished number therefore waits for nothing that is not
// there, and blocks that run are not taken off the chip before they end.  The
// words are cleared to a pattern that no block writes by a kernel before.
//
// 1 - a^2 is b (2 - b) with b = 1 - a from its series where v is small: long
// memories have v of 1e-3 and less.  fp32 tensors also take h - b h instead of
// a h there (a rounds to 2^-25, which a memory of n tokens adds up n times).
#include <initializer_list>

#include "gated_scan_launch.h"
#include "lm_grid.h"
#include "ssm_device.h"

namespace ssm66 {
namespace gated_scan {

namespace {

constexpr int kGroup = 32;                     // chunks from one published state to the next
constexpr uint64_t kEmpty = ~(uint64_t)0;      // a word that is not there yet
constexpr float kCut = __builtin_inff();       // V of a stretch where a document starts

// ---- the gates ----------------------------------------------------------------

// e^x; PRECISE: the argument's product with log2 e in two parts (for finite e^x)
template <bool PRECISE>
__device__ __forceinline__ float exp_f(float x) {
  const float hi = x * kLog2e;
  const float e = exp2_hw(hi);
  if (!PRECISE) return e;
  const float lo = fmaf(x, 1.9259629911266175e-8f, fmaf(x, kLog2e, -hi));
  return fmaf(e * kLn2, lo, e);
}

// within what e^x can hold (a NaN stays one)
__device__ __forceinline__ float held(float x) { return x > 87.0f ? 87.0f : x < -87.0f ? -87.0f : x; }

// sigmoid(z) and 1 - sigmoid(z), both to a few units in the last place
template <bool PRECISE>
__device__ __forceinline__ void sigmoid2(float z, float* s, float* rest) {
  const float e = exp_f<PRECISE>(held(-z));
  *s = rcp_hw(1.0f + e);
  *rest = e * *s;
}
template <bool PRECISE>
__device__ __forceinline__ float sigmoid1(float z) {
  return rcp_hw(1.0f + exp_f<PRECISE>(PRECISE ? held(-z) : -z));
}

// 1 - e^-v from v and a = e^-v: the series where it leaves out less than half a
// unit (its last term), the difference above, where it has lost at most a bit
template <bool PRECISE>
__device__ __forceinline__ float one_minus(float v, float a) {
  if (PRECISE) {
    float s = fmaf(v, -1.0f / 3628800.0f, 1.0f / 362880.0f);
    s = fmaf(v, -s, 1.0f / 40320.0f);
    s = fmaf(v, -s, 1.0f / 5040.0f);
    s = fmaf(v, -s, 1.0f / 720.0f);
    s = fmaf(v, -s, 1.0f / 120.0f);
    s = fmaf(v, -s, 1.0f / 24.0f);
    s = fmaf(v, -s, 1.0f / 6.0f);
    s = fmaf(v, -s, 0.5f);
    s = fmaf(v, -s, 1.0f);
    return v < 0.6931472f ? v * s : 1.0f - a;
  }
  float s = fmaf(v, -1.0f / 120.0f, 1.0f / 24.0f);
  s = fmaf(v, -s, 1.0f / 6.0f);
  s = fmaf(v, -s, 0.5f);
  s = fmaf(v, -s, 1.0f);
  return v < 0.125f ? v * s : 1.0f - a;
}

// The factor of a state: a itself, or (PRECISE, where a is near 1) -b with the
// sign bit set, which stands for 1 - b.
template <bool PRECISE>
__device__ __forceinline__ float factor(float v, float a, float b) {
  return PRECISE && v < 0.6931472f ? -b : a;
}
template <bool PRECISE>
__device__ __forceinline__ float times(float f, float h) {
  if (!PRECISE) return f * h;
  const float t = f * h;
  return __float_as_int(f) < 0 ? t + h : t;
}
template <bool PRECISE>
__device__ __forceinline__ float advance(float f, float h, float u) {
  const float t = fmaf(f, h, u);
  if (!PRECISE) return t;
  return __float_as_int(f) < 0 ? t + h : t;
}

// What a stretch does to a state, its factor instead of V (kCut: a document
// starts in it, nothing of the state before is read, a NaN neither).
template <bool PRECISE>
__device__ __forceinline__ float stretch_factor(float V) {
  if (V == kCut) return kCut;
  const float a = exp_f<PRECISE>(-V);
  return PRECISE ? factor<true>(V, a, one_minus<true>(V, a)) : a;
}
template <bool PRECISE>
__device__ __forceinline__ float over(float f, float h, float add) {
  return f == kCut ? add : advance<PRECISE>(f, h, add);
}

// V of two stretches together
__device__ __forceinline__ float joint(float V, float W) { return V == kCut || W == kCut ? kCut : V + W; }

// ---- memory -------------------------------------------------------------------

// VEC neighbouring channels as they lie in memory
template <typename T, int VEC> struct Raw;
template <> struct Raw<float, 1> {
  typedef float type;
  static __device__ __forceinline__ void get(type r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ type put(const float (&f)[1]) { return f[0]; }
};
template <> struct Raw<bf16_bits, 1> {
  typedef uint16_t type;
  static __device__ __forceinline__ void get(type r, float (&f)[1]) { f[0] = to_f32(r); }
  static __device__ __forceinline__ type put(const float (&f)[1]) {
    return __builtin_bit_cast(uint16_t, (__bf16)f[0]);
  }
};
template <> struct Raw<bf16_bits, 2> {
  typedef uint32_t type;
  static __device__ __forceinline__ void get(type r, float (&f)[2]) {
    f[0] = __uint_as_float(r << 16);
    f[1] = __uint_as_float(r & 0xffff0000u);
  }
  static __device__ __forceinline__ type put(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
};

__device__ __forceinline__ uint64_t word_of(float hi, float lo) {
  const uint64_t w = (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
  return w == kEmpty ? kEmpty - 1 : w;  // a NaN either way
}
__device__ __forceinline__ void publish(uint64_t* at, float hi, float lo) {
  __hip_atomic_store(at, word_of(hi, lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t look(const uint64_t* at) {
  return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float hi_of(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }
__device__ __forceinline__ float lo_of(uint64_t w) { return __uint_as_float((uint32_t)w); }

__global__ __launch_bounds__(256) void clear_kernel(uint32_t* ticket, uint64_t* words, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * 256;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += step) words[k] = kEmpty;
}

// Which tokens and channels a thread has.  `at`: 0, 1, ... of the chunks in the
// order they are taken (from the end backwards).
template <int VEC, int TOK, int W>
struct Spot {
  int at, chunk, lane, w;
  int64_t b, t0;
  int c;
  bool here;
  int real, inside;  // of the wave's tokens, those before the length and before L
  uint32_t cuts;     // bit j: a document starts at the wave's token j

  __device__ __forceinline__ Spot(const Args& p, uint32_t n, bool backward) {
    const uint32_t rows = p.blocks / (uint32_t)p.chunks;
    at = (int)(n / rows);
    const uint32_t row = n % rows;
    b = row / (uint32_t)p.tiles;
    chunk = backward ? p.chunks - 1 - at : at;
    lane = (int)threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    c = ((int)(row % (uint32_t)p.tiles) * 64 + lane) * VEC;
    here = c < p.dim;
    t0 = (int64_t)chunk * (TOK * W) + w * TOK;
    int64_t len = p.L;
    if (p.seq_lens) {
      len = p.seq_lens[b];
      len = len < 0 ? 0 : len > p.L ? p.L : len;
    }
    const int64_t left = len - t0, out = p.L - t0;
    real = left <= 0 ? 0 : left >= TOK ? TOK : (int)left;
    inside = out <= 0 ? 0 : out >= TOK ? TOK : (int)out;
    cuts = 0;
    if (p.reset && real > 0) {
      const bool start = lane < real && p.reset[b * p.L + t0 + lane] != 0;
      cuts = (uint32_t)__ballot(start);
    }
  }
  __device__ __forceinline__ int64_t offset(const Args& p) const { return (b * p.L + t0) * p.dim + c; }
};

// The wave's tokens of one tensor; what is not there is zero.
template <typename T, int VEC, int TOK, int W>
__device__ __forceinline__ void load_tokens(const Args& p, const Spot<VEC, TOK, W>& s, const void* from,
                                            typename Raw<T, VEC>::type (&raw)[TOK]) {
  typedef typename Raw<T, VEC>::type R;
  const T* const at = (const T*)from + s.offset(p);
  if (s.real == TOK && s.here) {
#pragma unroll
    for (int j = 0; j < TOK; ++j) raw[j] = *(const R*)(at + (int64_t)j * p.dim);
  } else {
#pragma unroll
    for (int j = 0; j < TOK; ++j)
      raw[j] = s.here && j < s.real ? *(const R*)(at + (int64_t)j * p.dim) : (R)0;
  }
}

// ---- the chunks before a block's own --------------------------------------------
//
// Called by all threads of a block between two barriers: wave w joins its share
// of the words and leaves (factor, H) in `joined`; the wave behind the last
// word's returns the state before the group, through `start`.

template <bool PRECISE, int VEC, int W>
__device__ __forceinline__ void join_before(const Args& p, int at, int64_t row0, bool here, int w,
                                            int lane, float2* joined, float* start) {
  const int first = at / kGroup * kGroup, n = at - first;
  const int64_t stride = p.batch * (int64_t)p.dim;
  constexpr int kShare = (kGroup + W - 1) / W;  // chunks of a wave
  if (here) {
    float V[VEC], H[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) V[k] = H[k] = 0.0f;
    const int64_t base = (int64_t)(first + w * kShare) * stride + row0;
    uint64_t word[kShare][VEC];
#pragma unroll
    for (int q = 0; q < kShare; ++q)
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        word[q][k] = w * kShare + q < n ? look(p.sums + base + q * stride + k) : 0;
#pragma unroll
    for (int q = 0; q < kShare; ++q) {
      if (w * kShare + q >= n) break;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        while (word[q][k] == kEmpty) {
          __builtin_amdgcn_s_sleep(1);
          word[q][k] = look(p.sums + base + q * stride + k);
        }
        const float f = stretch_factor<PRECISE>(hi_of(word[q][k]));
        H[k] = over<PRECISE>(f, H[k], lo_of(word[q][k]));
        V[k] = joint(V[k], hi_of(word[q][k]));
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      joined[w * (64 * VEC) + lane * VEC + k] = make_float2(stretch_factor<PRECISE>(V[k]), H[k]);
    if (w == W - 1 && first > 0) {
      const uint64_t* const g = p.groups + (int64_t)(first / kGroup - 1) * stride + row0;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        uint64_t s = look(g + k);
        while (s == kEmpty) {
          __builtin_amdgcn_s_sleep(1);
          s = look(g + k);
        }
        start[lane * VEC + k] = lo_of(s);
      }
    }
  }
}

// The block's number.
template <bool MANY>
__device__ __forceinline__ uint32_t block_number(const Args& p) {
  if (!MANY) return blockIdx.y * gridDim.x + blockIdx.x;
  __shared__ uint32_t number;
  if (threadIdx.x == 0)
    number = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(number);
}

// ---- forwards -----------------------------------------------------------------

template <typename T, int VEC, int TOK, int W, bool MANY>
__global__ __launch_bounds__(64 * W, 4) void fwd_kernel(const Args p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  typedef Raw<T, VEC> IO;
  __shared__ float2 pair[W * 64 * VEC], joined[W * 64 * VEC];
  __shared__ float vsum[W * 64 * VEC], start[64 * VEC];
  const uint32_t n = block_number<MANY>(p);
  if (n >= p.blocks) return;
  const Spot<VEC, TOK, W> s(p, n, false);
  const int64_t row = s.b * p.dim + s.c;

  typename IO::type rx[TOK], rr[TOK], ri[TOK];
  load_tokens<T>(p, s, p.r, rr);
  load_tokens<T>(p, s, p.i, ri);
  load_tokens<T>(p, s, p.x, rx);
  float d[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) d[k] = s.here ? p.decay[s.c + k] : 0.0f;

  float f[TOK][VEC], u[TOK][VEC], V[VEC], H[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) V[k] = H[k] = 0.0f;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    float x[VEC], r[VEC], i[VEC];
    IO::get(rx[j], x);
    IO::get(rr[j], r);
    IO::get(ri[j], i);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float v = d[k] * sigmoid1<PRECISE>(r[k]);
      const float a = exp_f<PRECISE>(-v);
      const float b = one_minus<PRECISE>(v, a);
      f[j][k] = factor<PRECISE>(v, a, b);
      u[j][k] = __builtin_amdgcn_sqrtf(b * (2.0f - b)) * sigmoid1<PRECISE>(i[k]) * x[k];
      if (j < s.real) V[k] += v;
    }
  }
  const bool plain = s.real == TOK && s.cuts == 0;  // the whole wave alike
  if (plain) {
#pragma unroll
    for (int j = 0; j < TOK; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) H[k] = advance<PRECISE>(f[j][k], H[k], u[j][k]);
  } else {
#pragma unroll
    for (int j = 0; j < TOK; ++j)
      if (j < s.real) {
        const bool cut = s.cuts >> j & 1;
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          H[k] = cut ? u[j][k] : advance<PRECISE>(f[j][k], H[k], u[j][k]);
      }
    if (s.cuts)
#pragma unroll
      for (int k = 0; k < VEC; ++k) V[k] = kCut;
  }
  const int slot = s.w * (64 * VEC) + s.lane * VEC;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    pair[slot + k] = make_float2(stretch_factor<PRECISE>(V[k]), H[k]);
    vsum[slot + k] = V[k];
  }
  lds_barrier();

  float h[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) h[k] = s.here && p.h0 ? p.h0[row + k] : 0.0f;
  if (MANY) {
    const int first = s.at / kGroup * kGroup;
    if (s.w == 0 && s.here && s.at + 1 < p.chunks && s.at + 1 < first + kGroup) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float Vb = 0.0f, Hb = 0.0f;
#pragma unroll
        for (int q = 0; q < W; ++q) {
          const float2 e = pair[q * (64 * VEC) + s.lane * VEC + k];
          Hb = over<PRECISE>(e.x, Hb, e.y);
          Vb = joint(Vb, vsum[q * (64 * VEC) + s.lane * VEC + k]);
        }
        publish(p.sums + (int64_t)s.at * (p.batch * p.dim) + row + k, Vb, Hb);
      }
    }
    join_before<PRECISE, VEC, W>(p, s.at, row, s.here, s.w, s.lane, joined, start);
    lds_barrier();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if (first > 0) h[k] = start[s.lane * VEC + k];
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float2 e = joined[q * (64 * VEC) + s.lane * VEC + k];
        h[k] = over<PRECISE>(e.x, h[k], e.y);
      }
    }
  }
  if (s.w == 0 && s.here && p.states)
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      p.states[(s.b * p.chunks + s.chunk) * p.dim + s.c + k] = h[k];
  for (int q = 0; q < s.w; ++q)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float2 e = pair[q * (64 * VEC) + s.lane * VEC + k];
      h[k] = over<PRECISE>(e.x, h[k], e.y);
    }

  typename IO::type* out = (typename IO::type*)((T*)p.y + s.offset(p));
  if (plain) {
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) h[k] = advance<PRECISE>(f[j][k], h[k], u[j][k]);
      if (s.here) *(typename IO::type*)((T*)out + (int64_t)j * p.dim) = IO::put(h);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
      const bool cut = s.cuts >> j & 1;
      float o[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (j < s.real) h[k] = cut ? u[j][k] : advance<PRECISE>(f[j][k], h[k], u[j][k]);
        o[k] = j < s.real ? h[k] : 0.0f;
      }
      if (s.here && j < s.inside) *(typename IO::type*)((T*)out + (int64_t)j * p.dim) = IO::put(o);
    }
  }
  if (s.w == W - 1 && s.here) {
    if (MANY && s.at % kGroup == kGroup - 1 && s.at + 1 < p.chunks)
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        publish(p.groups + (int64_t)(s.at / kGroup) * (p.batch * p.dim) + row + k, 0.0f, h[k]);
    if (p.last_state && s.chunk == p.chunks - 1)
#pragma unroll
      for (int k = 0; k < VEC; ++k) p.last_state[row + k] = h[k];
  }
}

// ---- backwards ----------------------------------------------------------------
//
// A block computes its gates and, from the state before its chunk, its states
// again; the adjoint comes from the right as the state does from the left.

template <typename T, int VEC, int TOK, int W, bool MANY>
__global__ __launch_bounds__(64 * W, 4) void bwd_kernel(const Args p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  typedef Raw<T, VEC> IO;
  // (factor, H) forwards and D, what a stretch adds to the adjoint, of each wave
  __shared__ float2 pair[W * 64 * VEC], joined[W * 64 * VEC];
  __shared__ float back[W * 64 * VEC], vsum[W * 64 * VEC], start[64 * VEC];
  const uint32_t n = block_number<MANY>(p);
  if (n >= p.blocks) return;
  const Spot<VEC, TOK, W> s(p, n, true);
  const int64_t row = s.b * p.dim + s.c;

  typename IO::type rx[TOK], rr[TOK], ri[TOK], rd[TOK];
  load_tokens<T>(p, s, p.r, rr);
  load_tokens<T>(p, s, p.i, ri);
  load_tokens<T>(p, s, p.x, rx);
  load_tokens<T>(p, s, p.dy, rd);
  float d[VEC], h[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    d[k] = s.here ? p.decay[s.c + k] : 0.0f;
    h[k] = s.here && p.states ? p.states[(s.b * p.chunks + s.chunk) * p.dim + s.c + k] : 0.0f;
  }

  float f[TOK][VEC], u[TOK][VEC], m[TOK][VEC], V[VEC], H[VEC], D[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) V[k] = H[k] = D[k] = 0.0f;
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    float x[VEC], r[VEC], i[VEC];
    IO::get(rx[j], x);
    IO::get(rr[j], r);
    IO::get(ri[j], i);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float v = d[k] * sigmoid1<PRECISE>(r[k]);
      const float a = exp_f<PRECISE>(-v);
      const float b = one_minus<PRECISE>(v, a);
      f[j][k] = factor<PRECISE>(v, a, b);
      m[j][k] = __builtin_amdgcn_sqrtf(b * (2.0f - b));
      u[j][k] = m[j][k] * sigmoid1<PRECISE>(i[k]) * x[k];
      if (j < s.real) V[k] += v;
    }
  }
  const bool plain = s.real == TOK && s.cuts == 0;
  if (plain) {
#pragma unroll
    for (int j = 0; j < TOK; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) H[k] = advance<PRECISE>(f[j][k], H[k], u[j][k]);
#pragma unroll
    for (int j = TOK - 1; j >= 0; --j) {
      float dy[VEC];
      IO::get(rd[j], dy);
#pragma unroll
      for (int k = 0; k < VEC; ++k) D[k] = times<PRECISE>(f[j][k], dy[k] + D[k]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < TOK; ++j)
      if (j < s.real) {
        const bool cut = s.cuts >> j & 1;
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          H[k] = cut ? u[j][k] : advance<PRECISE>(f[j][k], H[k], u[j][k]);
      }
#pragma unroll
    for (int j = TOK - 1; j >= 0; --j)
      if (j < s.real) {
        const bool cut = s.cuts >> j & 1;
        float dy[VEC];
        IO::get(rd[j], dy);
#pragma unroll
        for (int k = 0; k < VEC; ++k) D[k] = cut ? 0.0f : times<PRECISE>(f[j][k], dy[k] + D[k]);
      }
    if (s.cuts)
#pragma unroll
      for (int k = 0; k < VEC; ++k) V[k] = kCut;
  }
  const int slot = s.w * (64 * VEC) + s.lane * VEC;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    pair[slot + k] = make_float2(stretch_factor<PRECISE>(V[k]), H[k]);
    back[slot + k] = D[k];
    vsum[slot + k] = V[k];
  }
  lds_barrier();

  float c[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) c[k] = s.here && p.dlast ? p.dlast[row + k] : 0.0f;
  if (MANY) {
    const int first = s.at / kGroup * kGroup;
    if (s.w == 0 && s.here && s.at + 1 < p.chunks && s.at + 1 < first + kGroup) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float Vb = 0.0f, Db = 0.0f;
#pragma unroll
        for (int q = W - 1; q >= 0; --q) {
          const int o = q * (64 * VEC) + s.lane * VEC + k;
          Db = over<PRECISE>(pair[o].x, Db, back[o]);
          Vb = joint(Vb, vsum[o]);
        }
        publish(p.sums + (int64_t)s.at * (p.batch * p.dim) + row + k, Vb, Db);
      }
    }
    join_before<PRECISE, VEC, W>(p, s.at, row, s.here, s.w, s.lane, joined, start);
    lds_barrier();
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      if (first > 0) c[k] = start[s.lane * VEC + k];
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float2 e = joined[q * (64 * VEC) + s.lane * VEC + k];
        c[k] = over<PRECISE>(e.x, c[k], e.y);
      }
    }
  }
  for (int q = 0; q < s.w; ++q)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float2 e = pair[q * (64 * VEC) + s.lane * VEC + k];
      h[k] = over<PRECISE>(e.x, h[k], e.y);
    }
  for (int q = W - 1; q > s.w; --q)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int o = q * (64 * VEC) + s.lane * VEC + k;
      c[k] = over<PRECISE>(pair[o].x, c[k], back[o]);
    }

  // the gates are computed again rather than kept: what the compiler may not
  // know to be the same words as above
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    asm volatile("" : "+v"(rr[j]));
    asm volatile("" : "+v"(ri[j]));
    asm volatile("" : "+v"(rx[j]));
    asm volatile("" : "+v"(rd[j]));
  }
  // the states before each token, in the place of what the tokens add
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const bool cut = s.cuts >> j & 1;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float before = cut ? 0.0f : h[k];
      if (j < s.real) h[k] = cut ? u[j][k] : advance<PRECISE>(f[j][k], h[k], u[j][k]);
      u[j][k] = before;
    }
  }
  float P[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) P[k] = 0.0f;
  const int64_t at = s.offset(p);
#pragma unroll
  for (int j = TOK - 1; j >= 0; --j) {
    float x[VEC], r[VEC], i[VEC], dy[VEC], dx[VEC], dr[VEC], di[VEC];
    IO::get(rx[j], x);
    IO::get(rr[j], r);
    IO::get(ri[j], i);
    IO::get(rd[j], dy);
    const bool real = j < s.real, cut = s.cuts >> j & 1;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float sr, rest_r, g, rest_g;
      sigmoid2<PRECISE>(r[k], &sr, &rest_r);
      sigmoid2<PRECISE>(i[k], &g, &rest_g);
      const float v = d[k] * sr, lam = dy[k] + c[k];
      const float al = times<PRECISE>(f[j][k], lam);
      const float gx = g * x[k], lm = lam * m[j][k];
      // a v / m: 0 where v is (m is the root of about 2 v there)
      const float avm = times<PRECISE>(f[j][k], v * rcp_hw(fmaxf(m[j][k], 1e-30f)));
      const float q = fmaf(gx, avm, -v * u[j][k]) * al;
      dx[k] = real ? lm * g : 0.0f;
      di[k] = real ? lm * gx * rest_g : 0.0f;
      dr[k] = real ? q * rest_r : 0.0f;
      if (real) {
        P[k] += q;
        c[k] = cut ? 0.0f : al;
      }
    }
    if (s.here && j < s.inside) {
      *(typename IO::type*)((T*)p.dx + at + (int64_t)j * p.dim) = IO::put(dx);
      *(typename IO::type*)((T*)p.dr + at + (int64_t)j * p.dim) = IO::put(dr);
      *(typename IO::type*)((T*)p.di + at + (int64_t)j * p.dim) = IO::put(di);
    }
  }
  if (s.w == 0 && s.here) {
    if (MANY && s.at % kGroup == kGroup - 1 && s.at + 1 < p.chunks)
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        publish(p.groups + (int64_t)(s.at / kGroup) * (p.batch * p.dim) + row + k, 0.0f, c[k]);
    if (p.dh0 && s.chunk == 0)
#pragma unroll
      for (int k = 0; k < VEC; ++k) p.dh0[row + k] = c[k];
  }
  if (!p.part) return;
  lds_barrier();  // vsum has been read
#pragma unroll
  for (int k = 0; k < VEC; ++k) vsum[slot + k] = P[k];
  lds_barrier();
  if (s.w == 0 && s.here)
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float t = 0.0f;
#pragma unroll
      for (int q = 0; q < W; ++q) t += vsum[q * (64 * VEC) + s.lane * VEC + k];
      p.part[((int64_t)s.chunk * p.batch + s.b) * p.dim + s.c + k] = t;
    }
}

// ddecay from the rows of partial sums, added in fp64 in a fixed order: 64
// channels of a block, 16 waves that take every 16th row
__global__ __launch_bounds__(1024) void decay_sum_kernel(const float* part, const float* decay,
                                                         float* ddecay, int64_t rows, int dim) {
  __shared__ double sums[16][64];
  const int lane = (int)threadIdx.x & 63, w = (int)threadIdx.x >> 6;
  const int c = (int)blockIdx.x * 64 + lane;
  double t = 0.0;
  if (c < dim) {
    int64_t r = w;
    for (; r + 48 < rows; r += 64) {
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = part[(r + 16 * q) * dim + c];
#pragma unroll
      for (int q = 0; q < 4; ++q) t += v[q];
    }
    for (; r < rows; r += 16) t += part[r * dim + c];
  }
  sums[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < dim) {
    for (int q = 1; q < 16; ++q) t += sums[q][lane];
    ddecay[c] = (float)(t / (double)decay[c]);
  }
}

// ---- one token ----------------------------------------------------------------

template <typename T, int VEC>
__global__ __launch_bounds__(256) void step_kernel(const StepArgs p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  typedef Raw<T, VEC> IO;
  typedef typename IO::type R;
  const int64_t n = p.batch * p.dim / VEC, stride = (int64_t)gridDim.x * 256;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += stride) {
    const int64_t at = e * VEC;
    const int c = (int)(at % p.dim);
    float x[VEC], r[VEC], i[VEC], h[VEC];
    IO::get(*(const R*)((const T*)p.x + at), x);
    IO::get(*(const R*)((const T*)p.r + at), r);
    IO::get(*(const R*)((const T*)p.i + at), i);
#pragma unroll
    for (int k = 0; k < VEC; ++k) h[k] = p.state[at + k];
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float v = p.decay[c + k] * sigmoid1<PRECISE>(r[k]);
      const float a = exp_f<PRECISE>(-v);
      const float b = one_minus<PRECISE>(v, a);
      const float u = __builtin_amdgcn_sqrtf(b * (2.0f - b)) * sigmoid1<PRECISE>(i[k]) * x[k];
      h[k] = advance<PRECISE>(factor<PRECISE>(v, a, b), h[k], u);
      p.state[at + k] = h[k];
    }
    *(R*)((T*)p.y + at) = IO::put(h);
  }
}

// ---- launches -------------------------------------------------------------------

int64_t chunks_of(int64_t L) { return L > 0 ? (L + kChunk - 1) / kChunk : 1; }
int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

struct Layout { int64_t ticket, sums, groups, part, bytes; };
Layout layout(int64_t batch, int64_t L, int64_t dim, bool need_part) {
  const int64_t chunks = chunks_of(L), rows = batch * dim;
  Layout a = {};
  int64_t at = 0;
  if (chunks > 1) {
    a.ticket = at; at += 256;
    a.sums = at;   at += up(8 * chunks * rows);
    a.groups = at; at += up(8 * ((chunks + kGroup - 1) / kGroup) * rows);
  }
  a.part = at;
  if (need_part) at += up(4 * chunks * rows);
  a.bytes = at;
  return a;
}

void place(Args& p, int vec) {
  const Layout a = layout(p.batch, p.L, p.dim, p.ddecay != nullptr);
  char* const ws = (char*)p.ws;
  p.chunks = (int)chunks_of(p.L);
  p.tiles = (p.dim + 64 * vec - 1) / (64 * vec);
  p.blocks = (uint32_t)(p.batch * p.tiles * p.chunks);
  p.ticket = (uint32_t*)(ws + a.ticket);
  p.sums = (uint64_t*)(ws + a.sums);
  p.groups = (uint64_t*)(ws + a.groups);
  p.part = p.ddecay ? (float*)(ws + a.part) : nullptr;
}

hipError_t clear(const Args& p, hipStream_t s) {
  // the words of the chunks and of the groups lie side by side
  const int64_t n = (int64_t)(p.groups - p.sums) + ((int64_t)p.chunks + kGroup - 1) / kGroup * (p.batch * p.dim);
  const int64_t blocks = (n + 1023) / 1024;
  clear_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(p.ticket, p.sums, n);
  return hipGetLastError();
}

template <typename T, int VEC, int TOK, int W, bool BWD>
hipError_t launch(Args p, hipStream_t s) {
  static_assert(TOK * W == kChunk, "states are kept every kChunk tokens");
  place(p, VEC);
  const Grid g = grid_of(p.blocks, 64 * W);
  const dim3 grid(g.x, g.more), block(64 * W);
  if (p.chunks > 1) {
    const hipError_t e = clear(p, s);
    if (e != hipSuccess) return e;
    if constexpr (BWD) bwd_kernel<T, VEC, TOK, W, true><<<grid, block, 0, s>>>(p);
    else fwd_kernel<T, VEC, TOK, W, true><<<grid, block, 0, s>>>(p);
  } else {
    if constexpr (BWD) bwd_kernel<T, VEC, TOK, W, false><<<grid, block, 0, s>>>(p);
    else fwd_kernel<T, VEC, TOK, W, false><<<grid, block, 0, s>>>(p);
  }
  return hipGetLastError();
}

bool aligned4(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if ((uintptr_t)q % 4) return false;
  return true;
}

// two bf16 channels a thread where rows keep their words whole
bool pairs(int dim, std::initializer_list<const void*> ptrs) {
  return dim % 2 == 0 && dim > 64 && aligned4(ptrs);
}

}  // namespace

bool fits(int64_t batch, int64_t L, int64_t dim) {
  // block numbers are 32-bit, and so are chunk numbers and channels
  const __int128 blocks = (__int128)batch * ((dim + 63) / 64) * chunks_of(L);
  return dim <= (1 << 24) && chunks_of(L) < (1 << 24) && blocks < 0x7fffffff;
}

size_t workspace_bytes(int64_t batch, int64_t L, int64_t dim, bool backward, bool need_ddecay) {
  return (size_t)layout(batch, L, dim, backward && need_ddecay).bytes;
}

hipError_t forward(const Args& p, bool f32, hipStream_t s) {
  if (f32) return launch<float, 1, 16, 8, false>(p, s);
  if (pairs(p.dim, {p.x, p.r, p.i, p.y})) return launch<bf16_bits, 2, 16, 8, false>(p, s);
  return launch<bf16_bits, 1, 16, 8, false>(p, s);
}

hipError_t backward(const Args& p, bool f32, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.batch == 0) {
  } else if (f32) e = launch<float, 1, 8, 16, true>(p, s);
  else if (pairs(p.dim, {p.x, p.r, p.i, p.dy, p.dx, p.dr, p.di}))
    e = launch<bf16_bits, 2, 8, 16, true>(p, s);
  else e = launch<bf16_bits, 1, 8, 16, true>(p, s);
  if (e != hipSuccess || !p.ddecay) return e;
  const Layout a = layout(p.batch, p.L, p.dim, true);
  decay_sum_kernel<<<(p.dim + 63) / 64, 1024, 0, s>>>((const float*)((const char*)p.ws + a.part), p.decay,
                                                      p.ddecay, chunks_of(p.L) * p.batch, p.dim);
  return hipGetLastError();
}

hipError_t step(const StepArgs& p, bool f32, hipStream_t s) {
  const bool two = !f32 && p.dim % 2 == 0 && aligned4({p.x, p.r, p.i, p.y});
  const int64_t n = p.batch * p.dim / (two ? 2 : 1);
  const int64_t blocks = (n + 255) / 256;
  const unsigned g = (unsigned)(blocks < 8192 ? blocks : 8192);
  if (f32) step_kernel<float, 1><<<g, 256, 0, s>>>(p);
  else if (two) step_kernel<bf16_bits, 2><<<g, 256, 0, s>>>(p);
  else step_kernel<bf16_bits, 1><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace gated_scan
}  // namespace ssm66
