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
// One pass over the tensors.  A block takes 128 tokens (64 backwards) of a tile of
// 64 or 128 channels, a wave 8 or 16 of the tokens, a thread one or two channels of
// them in registers, so that the recurrence itself is a chain of multiply-adds.
// What a stretch of tokens does to a state is the pair (V, H): h -> exp(-V) h + H,
// V the sum of its v.  Pairs are joined over the waves in LDS and over the chunks
// through memory: a block publishes the pair of its chunk as one 64-bit word, waits
// for the words of the chunks before it in its group of chunks and for the state
// before the group, and goes on with its tokens, which never left the registers.
// The order of every join is fixed by the chunk's number, so repeated calls give
// identical bits.
//
// Why the waits end: a block that has begun takes its chunk's number from a
// counter, chunks of every row in order, and waits only for words of smaller
// numbers of the same counter.  Of the numbers taken the smallest unfinished one
// waits for nothing that is not there, and blocks that run are not taken off the
// chip before they end.  The words are cleared to a pattern that no block writes
// by a kernel before.
//
// Measured (a copy reaches 5.1 TB/s), calls with inputs from HBM and the kernel that
// clears the words (2 to 3 us): 8 x 2048 x 1536, bf16, forwards 51 us (201 MB once,
// the kernel at 4.3 TB/s), backwards 93 (352 MB, its kernel at 4.2, the sums of
// ddecay 4.5); 65536 x 2048 forwards 233 (1074 MB at 4.6).  HBM bounds it, and in
// front of that a block's waits: for its loads, its number and the words of others
// it waits 5 of the 10 us of its life; the vector units are busy for 55% of the
// time forwards and 60% backwards.
// 3 x 1537 x 1000, fp32: the kernels 25 and 38 us for 14 and 25 of bytes.  Their
// blocks' chain is load, 72 and 121 instructions a value, join, store; forwards 624
// blocks are one round (768 run at a time), backwards 1200 are more than two (512).
//
// 1 - a^2 comes from its series where v is small: long memories have v of 1e-3 and
// less.  fp32 tensors also take h - (1 - a) h instead of a h there (a rounds to
// 2^-25, which a memory of n tokens adds up n times), and so do for bf16 tensors the
// step, the state after a sequence and the gradient of that before it: 16384 tokens of fixed gates with v
// of 2.5e-6 to 1e-5 leave a state of relative error 3.5e-6 as steps (with a h
// 2.8e-4), 4.0e-7 as calls of 64 (1.9e-5) and 2.3e-7 as one call.
#include "gated_scan_launch.h"
#include "lm_grid.h"
#include "vec_io.h"

namespace ssm66 {
namespace gated_scan {

namespace {

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

template <bool PRECISE>
__device__ __forceinline__ float sigmoid1(float z) {
  return rcp_hw(1.0f + exp_f<PRECISE>(PRECISE ? held(-z) : -z));
}
// sigmoid(z) and 1 - sigmoid(z), both to a few units in the last place.
__device__ __forceinline__ void sigmoid2(float z, float* s, float* rest) {
  const float e = exp_f<true>(held(-fabsf(z)));
  const float r = rcp_hw(1.0f + e), er = e * r;
  *s = z > 0.0f ? r : er;
  *rest = z > 0.0f ? er : r;
}
// Both of them in one number, of which the fraction is sigmoid(z) and that of its
// negative 1 - sigmoid(z): the smaller of the two, with the sign bit set where that
// is 1 - sigmoid(z).  The fraction of 0 is 0 and not 1, so 1 - sigmoid(z) is never 0;
// a gate of 0 (z below -88) has 0 for both, and everything they multiply is 0 there.
struct Open { float s, both; };
__device__ __forceinline__ Open open_of(float z) {
  const float e = exp_f<false>(-z), s = rcp_hw(1.0f + e), rest = fmaf(e, s, 1.17549435e-38f);
  float both = s > 0.5f ? -rest : s;  // (a NaN stays one)
  asm("" : "+v"(both));  // made here: else s and rest both wait for the gradients, in 16 registers more
  return Open{s, both};
}
__device__ __forceinline__ float open_part(float both) { return __builtin_amdgcn_fractf(both); }
__device__ __forceinline__ float shut_part(float both) { return __builtin_amdgcn_fractf(-both); }

// 1 - e^-v from v and a = e^-v: the series where it leaves out less than half a
// unit (its last term), the difference above, where it has lost at most a bit
__device__ __forceinline__ float one_minus(float v, float a) {
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

// What a token's gate r does: V is v in the unit of the sums (natural where
// PRECISE, of log2 else, so that a is one exp2), f the factor of the state, m
// the root of 1 - a^2.  f is a itself, or (LESS, where a is near 1) -b with the
// sign bit set, which stands for 1 - b: a rounds to 2^-25, which is 1% of b = 1 - a
// where that is 3e-6, and a state that is handed on from token to token in memory
// would forget that much too fast or too slowly.
struct Gate { float V, f, m, s, rest; };  // s, rest: of sigmoid(r); s not PRECISE: both (open_of)
// -b = 2^-V - 1 for V below 0.07
__device__ __forceinline__ float minus_b(float V) {
  float s = fmaf(V, -0.0096181291f, 0.055504109f);
  s = fmaf(V, s, -0.24022651f);
  return V * fmaf(V, -s, -kLn2);
}
template <bool PRECISE>
__device__ __forceinline__ float sum_unit(float decay) { return PRECISE ? decay : decay * kLog2e; }
template <bool PRECISE, bool LESS = PRECISE>
__device__ __forceinline__ Gate gate_of(float d, float r) {  // d: sum_unit(decay)
  Gate g;
  if (PRECISE) {
    sigmoid2(r, &g.s, &g.rest);
    g.V = d * g.s;
    const float a = exp_f<true>(-g.V), b = one_minus(g.V, a);
    g.f = g.V < 0.6931472f ? -b : a;
    g.m = __builtin_amdgcn_sqrtf(b * (2.0f - b));
  } else {
    // below v = 0.05 four terms of a series, of 1 - a^2 (which leave out 8e-7 of
    // it) or of 1 - a (5e-8); a's rounding is 6e-7 of the differences above
    const Open o = open_of(r);
    g.s = o.both;
    g.V = d * o.s;
    const bool small = g.V < 0.07f;
    const float a = exp2_hw(-g.V);
    float m2;
    if (LESS) {
      const float f = minus_b(g.V);
      g.f = small ? f : a;
      m2 = small ? f * (-2.0f - f) : fmaf(-a, a, 1.0f);
    } else {
      float s = fmaf(g.V, -0.15388844f, 0.44403291f);
      s = fmaf(g.V, s, -0.96090603f);
      s = fmaf(g.V, s, 1.38629436f);
      g.f = a;
      m2 = small ? g.V * s : fmaf(-a, a, 1.0f);
    }
    g.m = __builtin_amdgcn_sqrtf(m2);
  }
  return g;
}

// f h and f h + u; LESS: f with the sign bit set stands for 1 + f.  kept() takes
// the product with the finite h nearest to h, and then adds h or what is left of it
// (0 or an infinity): an infinite state stays one, where -b h + h would make it a
// NaN (fp32, forwards and backwards, without and with it: 3 x 1537 x 1000 26.4 + 44.1,
// 26.6 + 45.0 us; 8 x 2048 x 1536 90.5 + 155.1, 90.9 + 156.1).
__device__ __forceinline__ float kept(float f, float h, float u) {
  const float fin = __builtin_amdgcn_fmed3f(h, -3.402823466e38f, 3.402823466e38f), t = fmaf(f, fin, u);
  return t + (__float_as_int(f) < 0 ? h : h - fin);
}
template <bool LESS>
__device__ __forceinline__ float times(float f, float h) {
  return LESS ? kept(f, h, 0.0f) : f * h;
}
template <bool LESS>
__device__ __forceinline__ float advance(float f, float h, float u) {
  return LESS ? kept(f, h, u) : fmaf(f, h, u);
}

// What a stretch of tokens does to a state, its factor instead of V (kCut: a
// document starts in it, nothing of the state before is read, a NaN neither).
template <bool PRECISE, bool LESS = PRECISE>
__device__ __forceinline__ float stretch_factor(float V) {
  if (V == kCut) return kCut;
  // a stretch of nothing is the factor 1 (an infinite state passes it as it is)
  if (PRECISE) {
    const float a = exp_f<true>(-V);
    return V < 0.6931472f && V > 0.0f ? -one_minus(V, a) : a;
  }
  // never 0, which would make an infinite state a NaN: the least number there is,
  // which leaves 5e-7 of the largest finite state (of a V that is a NaN the stretch's
  // H is one too)
  const float a = fmaxf(exp2_hw(-V), 1.4e-45f);
  return LESS && V < 0.07f && V > 0.0f ? minus_b(V) : a;
}
template <bool LESS>
__device__ __forceinline__ float over(float f, float h, float add) {
  return f == kCut ? add : advance<LESS>(f, h, add);
}
// V of two stretches together
__device__ __forceinline__ float joint(float V, float W) { return V == kCut || W == kCut ? kCut : V + W; }

// ---- memory -------------------------------------------------------------------

// VEC neighbouring channels as they lie in memory: their type there (from any
// address of a value) and elsewhere
template <typename T, int VEC> struct Raw;
template <> struct Raw<float, 1> {
  typedef float type, mem;
  static __device__ __forceinline__ void get(type r, float (&f)[1]) { f[0] = r; }
  static __device__ __forceinline__ type put(const float (&f)[1]) { return f[0]; }
};
template <> struct Raw<bf16_bits, 1> {
  typedef uint16_t type, mem;
  static __device__ __forceinline__ void get(type r, float (&f)[1]) { f[0] = to_f32(r); }
  static __device__ __forceinline__ type put(const float (&f)[1]) {
    return __builtin_bit_cast(uint16_t, (__bf16)f[0]);
  }
};
template <> struct Raw<bf16_bits, 2> {
  typedef uint32_t type;
  typedef uint32_t mem __attribute__((aligned(2)));
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

constexpr int kLine = 32;           // numbers from one counter to the next: 128 bytes
constexpr uint32_t kCounters = 128;  // at most

// the counters to 0, n words (an even number, from a 16-byte boundary on) to kEmpty
__global__ __launch_bounds__(256) void clear_kernel(uint32_t* tickets, uint32_t counters,
                                                    uint64_t* words, int64_t n) {
  const int64_t step = (int64_t)gridDim.x * 256;
  if (blockIdx.x == 0 && threadIdx.x < counters) tickets[threadIdx.x * kLine] = 0;
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n / 2; k += step)
    ((ulonglong2*)words)[k] = make_ulonglong2(kEmpty, kEmpty);
}

// The tile a block works on: a row (a tile of channels of one entry) and the
// number of its chunk, in the order they are taken.
struct Tile {
  uint32_t row;
  int at;
  bool real;
};
// The rows are dealt out to the counters and a block asks that of its number.  Of
// a counter's numbers the first belong to its rows' first chunks, and so on; a
// block waits for smaller numbers of its own counter.
template <bool MANY>
__device__ __forceinline__ Tile take_tile(const Args& p) {
  const uint32_t block = blockIdx.y * gridDim.x + blockIdx.x;
  if (!MANY) return Tile{block, 0, block < p.rows};
  if (block >= p.blocks) return Tile{0, 0, false};
  __shared__ uint32_t number;
  const uint32_t g = (uint32_t)__builtin_amdgcn_readfirstlane((int)(block % p.counters));
  if (threadIdx.x == 0)
    number = __hip_atomic_fetch_add(p.tickets + g * kLine, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const uint32_t n = (uint32_t)__builtin_amdgcn_readfirstlane((int)number);
  const uint32_t mine = (p.rows - g + p.counters - 1) / p.counters;  // rows of this counter
  const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane((int)(n / mine));
  return Tile{g + (n - at * mine) * p.counters, (int)at, at < (uint32_t)p.chunks};
}

// Which tokens and channels a thread has.  `at`: 0, 1, ... of the chunks in the
// order they are taken (from the end backwards).
template <int VEC, int TOK, int W>
struct Spot {
  int at, chunk, lane, w;
  int64_t b, t0;
  int c;
  bool here;
  int last;          // from t0 to the last token that may be read (negative past it)
  int real, inside;  // of the wave's tokens, those before the length and before L
  uint32_t cuts;     // bit j: a document starts at the wave's token j

  __device__ __forceinline__ Spot(const Args& p, const Tile& t, bool backward) {
    at = t.at;
    // a quotient comes from the vector unit; the rest is to stay on the scalar one
    const int entry = __builtin_amdgcn_readfirstlane((int)(t.row / (uint32_t)p.tiles));
    b = entry;
    chunk = backward ? p.chunks - 1 - at : at;
    lane = (int)threadIdx.x & 63;
    w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    c = ((int)(t.row - (uint32_t)entry * (uint32_t)p.tiles) * 64 + lane) * VEC;
    here = c < p.dim;
    // an odd number of channels: the last thread has the one before it too, and
    // what two threads have they compute and store alike
    if (VEC > 1 && here && c > p.dim - VEC) c = p.dim - VEC;
    t0 = (int64_t)chunk * (TOK * W) + w * TOK;
    int64_t len = p.L;
    if (p.seq_lens) {
      len = __builtin_amdgcn_readfirstlane(p.seq_lens[b]);
      len = len < 0 ? 0 : len > p.L ? p.L : len;
    }
    const int64_t left = len - t0, out = p.L - t0;
    real = left <= 0 ? 0 : left >= TOK ? TOK : (int)left;
    inside = out <= 0 ? 0 : out >= TOK ? TOK : (int)out;
    last = left > TOK ? TOK - 1 : left < 1 ? (int)((len > 0 ? len - 1 : 0) - t0) : (int)left - 1;
    cuts = 0;
  }
  __device__ __forceinline__ void read_cuts(const Args& p) {
    if (!p.reset || real <= 0) return;
    const bool start = lane < real && p.reset[b * p.L + t0 + lane] != 0;
    cuts = (uint32_t)__ballot(start);
  }
  // A tensor's rows of the wave: a scalar base and 32-bit offsets, that of row j
  // to be loaded and to be stored.  In the place of a token that is not there
  // the last real one is loaded, and the first channel: loads without a branch,
  // and what is made of them is left out of the sums and not stored.
  template <typename T>
  __device__ __forceinline__ const char* from(const Args& p, const void* t) const {
    return (const char*)t + ((b * p.L + t0 + (last < 0 ? last : 0)) * p.dim) * (int64_t)sizeof(T);
  }
  template <typename T>
  __device__ __forceinline__ uint32_t load_at(const Args& p, int j) const {
    const int q = j < last ? j : last < 0 ? 0 : last;
    return (here ? (uint32_t)c * (uint32_t)sizeof(T) : 0u) + (uint32_t)q * ((uint32_t)p.dim * (uint32_t)sizeof(T));
  }
  template <typename T>
  __device__ __forceinline__ char* to(const Args& p, void* t) const {
    return (char*)t + ((b * p.L + t0) * p.dim) * (int64_t)sizeof(T);
  }
  template <typename T>
  __device__ __forceinline__ uint32_t store_at(const Args& p, int j) const {
    return (uint32_t)c * (uint32_t)sizeof(T) + (uint32_t)j * ((uint32_t)p.dim * (uint32_t)sizeof(T));
  }
};

// ---- the chunks before a block's own --------------------------------------------

// Whether chunk `at` is the last of its group, and there are more: it publishes
// the state behind it, the others (but the last of all, whom nobody reads) their
// own word.
__device__ __forceinline__ bool ends_group(const Args& p, int at) {
  return (at & (p.group - 1)) == p.group - 1 && at + 1 < p.chunks;
}
__device__ __forceinline__ bool has_word(const Args& p, int at) {
  return (at & (p.group - 1)) != p.group - 1 && at + 1 < p.chunks;
}

// The state before chunk `at` of its row in the order of the chunks, by one
// wave: the words of the chunks between its group's start and itself, joined,
// over the state before the group (`begin`: before the first).  The chain from
// group to group is what a long row waits for, so nothing but one step stands
// between a group's state and the next one's.
template <bool PRECISE, int VEC>
__device__ __forceinline__ void state_before(const Args& p, int at, int64_t row0,
                                             const float (&begin)[VEC], float (&h)[VEC]) {
  constexpr int kAhead = 3;  // words on their way at a time
  const int n = at & (p.group - 1), first = at - n;
  const int64_t stride = p.batch * (int64_t)p.dim;
  const uint64_t* const group = p.groups + (int64_t)(first / p.group - 1) * stride + row0;
  uint64_t state[VEC];
  float V[VEC], H[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    state[k] = first > 0 ? look(group + k) : 0;
    V[k] = H[k] = 0.0f;
  }
  for (int q0 = 0; q0 < n; q0 += kAhead) {
    const uint64_t* const sums = p.sums + (int64_t)(first + q0) * stride + row0;
    uint64_t word[kAhead][VEC];
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int k = 0; k < VEC; ++k) word[q][k] = q0 + q < n ? look(sums + q * stride + k) : 0;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      if (q0 + q >= n) break;
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        while (word[q][k] == kEmpty) {
          __builtin_amdgcn_s_sleep(1);
          word[q][k] = look(sums + q * stride + k);
        }
        H[k] = over<PRECISE>(stretch_factor<PRECISE>(hi_of(word[q][k])), H[k], lo_of(word[q][k]));
        V[k] = joint(V[k], hi_of(word[q][k]));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float f = stretch_factor<PRECISE>(V[k]);
    while (state[k] == kEmpty) {
      __builtin_amdgcn_s_sleep(1);
      state[k] = look(group + k);
    }
    h[k] = over<PRECISE>(f, first > 0 ? lo_of(state[k]) : begin[k], H[k]);
  }
}

// H of the wave's tokens, from a state of zero (or of `h`).
template <bool PRECISE, bool PLAIN, int VEC, int TOK>
__device__ __forceinline__ void run_tokens(int real, uint32_t cuts, const float (&f)[TOK][VEC],
                                           const float (&u)[TOK][VEC], float (&h)[VEC]) {
#pragma unroll
  for (int j = 0; j < TOK; ++j)
    if (PLAIN || j < real)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float t = advance<PRECISE>(f[j][k], h[k], u[j][k]);
        h[k] = !PLAIN && (cuts >> j & 1) ? u[j][k] : t;
      }
}

// What the wave's tokens add to the adjoint from their right.
template <typename T, bool PLAIN, int VEC, int TOK>
__device__ __forceinline__ void run_back(int real, uint32_t cuts, const float (&f)[TOK][VEC],
                                         const typename Raw<T, VEC>::type (&rd)[TOK], float (&c)[VEC]) {
#pragma unroll
  for (int j = TOK - 1; j >= 0; --j)
    if (PLAIN || j < real) {
      float dy[VEC];
      Raw<T, VEC>::get(rd[j], dy);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float t = times<sizeof(T) == 4>(f[j][k], dy[k] + c[k]);
        c[k] = !PLAIN && (cuts >> j & 1) ? 0.0f : t;
      }
    }
}

// The states before each token, in the place of what the tokens add; h: the
// state before the first.
template <bool PRECISE, bool PLAIN, int VEC, int TOK>
__device__ __forceinline__ void states_before(int real, uint32_t cuts, const float (&f)[TOK][VEC],
                                              float (&u)[TOK][VEC], float (&h)[VEC]) {
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    const bool cut = !PLAIN && (cuts >> j & 1);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float add = u[j][k];
      u[j][k] = cut ? 0.0f : h[k];
      const float t = advance<PRECISE>(f[j][k], h[k], add);
      if (PLAIN || j < real) h[k] = cut ? add : t;
    }
  }
}

// ---- forwards -----------------------------------------------------------------
//
// Between the two barriers wave 0 joins the block's waves (what stands before
// each of them, and the block's own word) while wave 1 looks at the chunks
// before.

template <typename T, int VEC, int TOK, int W, bool MANY>
__global__ __launch_bounds__(64 * W, 4) void fwd_kernel(const Args p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  constexpr int N = 64 * VEC;
  typedef Raw<T, VEC> IO;
  // (V, H) of each wave, then (factor, H) of the waves before it, and the state
  // before the chunk
  __shared__ float2 pair[W][N], ahead[W][N];
  __shared__ float start[N];
  const Tile tile = take_tile<MANY>(p);
  if (!tile.real) return;
  Spot<VEC, TOK, W> s(p, tile, false);

  typename IO::type rx[TOK] = {}, rr[TOK] = {}, ri[TOK] = {};
  if (MANY || p.L > 0)
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
      rr[j] = *(const typename IO::mem*)(s.template from<T>(p, p.r) + s.template load_at<T>(p, j));
      ri[j] = *(const typename IO::mem*)(s.template from<T>(p, p.i) + s.template load_at<T>(p, j));
      rx[j] = *(const typename IO::mem*)(s.template from<T>(p, p.x) + s.template load_at<T>(p, j));
    }
  s.read_cuts(p);
  const int64_t row = s.b * p.dim + s.c;
  const int slot = s.lane * VEC;
  float d[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) d[k] = sum_unit<PRECISE>(s.here ? p.decay[s.c + k] : 0.0f);

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
      const Gate g = gate_of<PRECISE>(d[k], r[k]);
      f[j][k] = g.f;
      u[j][k] = g.m * sigmoid1<PRECISE>(i[k]) * x[k];
      V[k] += j < s.real ? g.V : 0.0f;
    }
  }
  const bool plain = s.real == TOK && s.cuts == 0;  // the whole wave alike
  if (plain) run_tokens<PRECISE, true>(s.real, s.cuts, f, u, H);
  else run_tokens<PRECISE, false>(s.real, s.cuts, f, u, H);
#pragma unroll
  for (int k = 0; k < VEC; ++k) pair[s.w][slot + k] = make_float2(s.cuts ? kCut : V[k], H[k]);
  lds_barrier();

  if (s.w == 0) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float Vb = 0.0f, Hb = 0.0f;
#pragma unroll 2
      for (int q = 0; q < W; ++q) {
        const float2 e = pair[q][slot + k];
        ahead[q][slot + k] = make_float2(stretch_factor<PRECISE>(Vb), Hb);
        Hb = over<PRECISE>(stretch_factor<PRECISE>(e.x), Hb, e.y);
        Vb = joint(Vb, e.x);
      }
      if (MANY && s.here && has_word(p, s.at))
        publish(p.sums + (int64_t)s.at * (p.batch * p.dim) + row + k, Vb, Hb);
    }
  }
  if (s.w == 1) {
    float begin[VEC], h[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) h[k] = begin[k] = s.here && p.h0 ? p.h0[row + k] : 0.0f;
    const bool ends = MANY && ends_group(p, s.at);
    float fb[VEC], Hb[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) fb[k] = Hb[k] = 0.0f;
    if (ends)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float Vb = 0.0f;
#pragma unroll 2
        for (int q = 0; q < W; ++q) {
          const float2 e = pair[q][slot + k];
          Hb[k] = over<PRECISE>(stretch_factor<PRECISE>(e.x), Hb[k], e.y);
          Vb = joint(Vb, e.x);
        }
        fb[k] = stretch_factor<PRECISE>(Vb);
      }
    if (s.here) {
      if (MANY) state_before<PRECISE, VEC>(p, s.at, row, begin, h);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (ends)
          publish(p.groups + (int64_t)(s.at / p.group) * (p.batch * p.dim) + row + k, 0.0f,
                  over<PRECISE>(fb[k], h[k], Hb[k]));
        start[slot + k] = h[k];
      }
      // the state after the last chunk: bf16 calls join it from the chunk's own pair, its
      // factor as what that is less than 1, for the tokens' rounded factors would add
      // up in a state that is handed on from call to call, and a call of one token is a
      // step (64 x 64 x 1024: 13.5 us as before; with all factors so, 16.9)
      if (!PRECISE && p.last_state && s.chunk == p.chunks - 1)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          float V = 0.0f, H = 0.0f;
#pragma unroll
          for (int q = 0; q < W; ++q) {
            const float2 e = pair[q][slot + k];
            H = over<PRECISE>(stretch_factor<PRECISE>(e.x), H, e.y);
            V = joint(V, e.x);
          }
          p.last_state[row + k] = over<true>(stretch_factor<PRECISE, true>(V), h[k], H);
        }
    }
  }
  lds_barrier();

  float h[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    const float2 e = ahead[s.w][slot + k];
    h[k] = over<PRECISE>(e.x, start[slot + k], e.y);
  }
  if (p.states && s.here && s.w * TOK % kKeep == 0 && s.t0 < p.L)
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      p.states[(s.b * p.kept + s.t0 / kKeep) * p.dim + s.c + k] = h[k];
  if (plain) {
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) h[k] = advance<PRECISE>(f[j][k], h[k], u[j][k]);
      if (s.here)
        *(typename IO::mem*)(s.template to<T>(p, p.y) + s.template store_at<T>(p, j)) = IO::put(h);
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
      if (s.here && j < s.inside)
        *(typename IO::mem*)(s.template to<T>(p, p.y) + s.template store_at<T>(p, j)) = IO::put(o);
    }
  }
  if (PRECISE && s.w == W - 1 && s.here && p.last_state && s.chunk == p.chunks - 1)
#pragma unroll
    for (int k = 0; k < VEC; ++k) p.last_state[row + k] = h[k];
}

// ---- backwards ----------------------------------------------------------------
//
// A block computes its gates and, from the state before its chunk, its states
// again; the adjoint comes from the right as the state does from the left.  The
// gates stay in registers, x and dy wait in LDS meanwhile.

// What a block keeps of a token's gates: f, m, sigmoid(r), sigmoid(i) and what is
// left of both to 1 (bf16: each two of them in one register, open_of).
template <bool PRECISE, int VEC, int TOK>
struct Gates {
  float f[TOK][VEC], m[TOK][VEC], r[TOK][VEC], i[TOK][VEC];
  float rest_r[PRECISE ? TOK : 1][VEC], rest_i[PRECISE ? TOK : 1][VEC];
};

// The gradients of the wave's tokens, from the last to the first; before[j] is
// the state before token j, c the adjoint from the right, P the sum of P_t.
template <typename T, bool PLAIN, int VEC, int TOK, int W>
__device__ __forceinline__ void token_gradients(
    const Args& p, const Spot<VEC, TOK, W>& s, const typename Raw<T, VEC>::type* stash,
    const Gates<sizeof(T) == 4, VEC, TOK>& gate,
    const float (&before)[TOK][VEC], const float (&decay)[VEC], float (&c)[VEC], float (&P)[VEC]) {
  constexpr bool PRECISE = sizeof(T) == 4;
  typedef Raw<T, VEC> IO;
  typedef typename IO::mem R;
#pragma unroll
  for (int j = TOK - 1; j >= 0; --j) {
    float x[VEC], dy[VEC], dx[VEC], dr[VEC], di[VEC];
    IO::get(stash[j * (64 * W)], x);
    IO::get(stash[(TOK + j) * (64 * W)], dy);
    const bool real = PLAIN || j < s.real, cut = !PLAIN && (s.cuts >> j & 1);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float f = gate.f[j][k], m = gate.m[j][k];
      const float sr = PRECISE ? gate.r[j][k] : open_part(gate.r[j][k]);
      const float g = PRECISE ? gate.i[j][k] : open_part(gate.i[j][k]);
      const float rest_r = PRECISE ? gate.rest_r[PRECISE ? j : 0][k] : shut_part(gate.r[j][k]);
      const float rest_g = PRECISE ? gate.rest_i[PRECISE ? j : 0][k] : shut_part(gate.i[j][k]);
      const float v = decay[k] * sr, lam = dy[k] + c[k];
      const float al = times<PRECISE>(f, lam);
      const float gx = g * x[k], lm = lam * m;
      // a v / m: 0 where v is (m is the root of about 2 v there)
      const float vm = v * rcp_hw(fmaxf(m, 1e-30f)), fvm = f * vm;
      const float avm = PRECISE && __float_as_int(f) < 0 ? fvm + vm : fvm;
      const float q = fmaf(gx, avm, -(v * before[j][k])) * al;
      dx[k] = real ? lm * g : 0.0f;
      di[k] = real ? lm * gx * rest_g : 0.0f;
      dr[k] = real ? q * rest_r : 0.0f;
      if (real) {
        P[k] += q;
        c[k] = cut ? 0.0f : al;
      }
    }
    if (s.here && (PLAIN || j < s.inside)) {
      *(R*)(s.template to<T>(p, p.dx) + s.template store_at<T>(p, j)) = IO::put(dx);
      *(R*)(s.template to<T>(p, p.dr) + s.template store_at<T>(p, j)) = IO::put(dr);
      *(R*)(s.template to<T>(p, p.di) + s.template store_at<T>(p, j)) = IO::put(di);
    }
  }
}

template <typename T, int VEC, int TOK, int W, bool MANY>
__global__ __launch_bounds__(64 * W, 4) void bwd_kernel(const Args p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  constexpr int N = 64 * VEC;
  typedef Raw<T, VEC> IO;
  // (V, H) of each wave, and D, what it adds to the adjoint; then the state
  // before each wave, and (factor, D) of the waves behind it
  __shared__ float2 pair[W][N], behind[W][N];
  __shared__ float back[W][N], first[W][N], start[N];
  // each thread's own x and dy: the registers are for the gates
  __shared__ typename IO::type stashes[2 * TOK * 64 * W];
  typename IO::type* const stash = stashes + threadIdx.x;
  const Tile tile = take_tile<MANY>(p);
  if (!tile.real) return;
  Spot<VEC, TOK, W> s(p, tile, true);

  typename IO::type rx[TOK] = {}, rr[TOK] = {}, ri[TOK] = {}, rd[TOK] = {};
  if (MANY || p.L > 0)
#pragma unroll
    for (int j = 0; j < TOK; ++j) {
      rr[j] = *(const typename IO::mem*)(s.template from<T>(p, p.r) + s.template load_at<T>(p, j));
      ri[j] = *(const typename IO::mem*)(s.template from<T>(p, p.i) + s.template load_at<T>(p, j));
      rx[j] = *(const typename IO::mem*)(s.template from<T>(p, p.x) + s.template load_at<T>(p, j));
      rd[j] = *(const typename IO::mem*)(s.template from<T>(p, p.dy) + s.template load_at<T>(p, j));
    }
  s.read_cuts(p);
  const int64_t row = s.b * p.dim + s.c;
  const int slot = s.lane * VEC;
  float decay[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) decay[k] = s.here ? p.decay[s.c + k] : 0.0f;

  Gates<PRECISE, VEC, TOK> gate;
  float u[TOK][VEC], V[VEC], H[VEC], D[VEC];
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
      const Gate g = gate_of<PRECISE>(sum_unit<PRECISE>(decay[k]), r[k]);
      gate.f[j][k] = g.f;
      gate.m[j][k] = g.m;
      gate.r[j][k] = g.s;
      float open;
      if (PRECISE) {
        gate.rest_r[PRECISE ? j : 0][k] = g.rest;
        sigmoid2(i[k], &open, &gate.rest_i[PRECISE ? j : 0][k]);
        gate.i[j][k] = open;
      } else {
        const Open o = open_of(i[k]);
        gate.i[j][k] = o.both;
        open = o.s;
      }
      u[j][k] = g.m * open * x[k];
      V[k] += j < s.real ? g.V : 0.0f;
    }
  }
#pragma unroll
  for (int j = 0; j < TOK; ++j) {
    stash[j * (64 * W)] = rx[j];
    stash[(TOK + j) * (64 * W)] = rd[j];
  }
  const bool plain = s.real == TOK && s.cuts == 0;
  if (plain) {
    run_tokens<PRECISE, true>(s.real, s.cuts, gate.f, u, H);
    run_back<T, true>(s.real, s.cuts, gate.f, rd, D);
  } else {
    run_tokens<PRECISE, false>(s.real, s.cuts, gate.f, u, H);
    run_back<T, false>(s.real, s.cuts, gate.f, rd, D);
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    pair[s.w][slot + k] = make_float2(s.cuts ? kCut : V[k], H[k]);
    back[s.w][slot + k] = D[k];
  }
  lds_barrier();

  // wave 0: the states before the waves; wave 1: what stands behind them, and
  // the block's own word; wave 2: the chunks behind
  if (s.w == 0) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float h = s.here && p.states ? p.states[(s.b * p.kept + s.t0 / kKeep) * p.dim + s.c + k] : 0.0f;
#pragma unroll 2
      for (int q = 0; q < W; ++q) {
        const float2 e = pair[q][slot + k];
        first[q][slot + k] = h;
        h = over<PRECISE>(stretch_factor<PRECISE>(e.x), h, e.y);
      }
    }
  }
  if (s.w == 1) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      float Vb = 0.0f, Db = 0.0f;
#pragma unroll 2
      for (int q = W - 1; q >= 0; --q) {
        const float Vq = pair[q][slot + k].x, Dq = back[q][slot + k];
        behind[q][slot + k] = make_float2(stretch_factor<PRECISE>(Vb), Db);
        Db = over<PRECISE>(stretch_factor<PRECISE>(Vq), Db, Dq);
        Vb = joint(Vb, Vq);
      }
      if (MANY && s.here && has_word(p, s.at))
        publish(p.sums + (int64_t)s.at * (p.batch * p.dim) + row + k, Vb, Db);
    }
  }
  if (s.w == 2) {
    float begin[VEC], c[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) c[k] = begin[k] = s.here && p.dlast ? p.dlast[row + k] : 0.0f;
    const bool ends = MANY && ends_group(p, s.at);
    float fb[VEC], Db[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) fb[k] = Db[k] = 0.0f;
    if (ends)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float Vb = 0.0f;
#pragma unroll 2
        for (int q = W - 1; q >= 0; --q) {
          const float Vq = pair[q][slot + k].x;
          Db[k] = over<PRECISE>(stretch_factor<PRECISE>(Vq), Db[k], back[q][slot + k]);
          Vb = joint(Vb, Vq);
        }
        fb[k] = stretch_factor<PRECISE>(Vb);
      }
    if (s.here) {
      if (MANY) state_before<PRECISE, VEC>(p, s.at, row, begin, c);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (ends)
          publish(p.groups + (int64_t)(s.at / p.group) * (p.batch * p.dim) + row + k, 0.0f,
                  over<PRECISE>(fb[k], c[k], Db[k]));
        start[slot + k] = c[k];
      }
      // the gradient of the first state, handed on from call to call as the last state
      // is (not unrolled: 26 registers more in short calls, 64 x 64 x 1024 22.5 -> 27.4 us)
      if (!PRECISE && p.dh0 && s.chunk == 0)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          float V = 0.0f, D = 0.0f;
#pragma unroll 1
          for (int q = W - 1; q >= 0; --q) {
            const float Vq = pair[q][slot + k].x;
            D = over<PRECISE>(stretch_factor<PRECISE>(Vq), D, back[q][slot + k]);
            V = joint(V, Vq);
          }
          p.dh0[row + k] = over<true>(stretch_factor<PRECISE, true>(V), c[k], D);
        }
    }
  }
  lds_barrier();
  float h[VEC], c[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    h[k] = first[s.w][slot + k];
    const float2 e = behind[s.w][slot + k];
    c[k] = over<PRECISE>(e.x, start[slot + k], e.y);
  }

  float P[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) P[k] = 0.0f;
  if (plain) {
    states_before<PRECISE, true>(s.real, s.cuts, gate.f, u, h);
    token_gradients<T, true>(p, s, stash, gate, u, decay, c, P);
  } else {
    states_before<PRECISE, false>(s.real, s.cuts, gate.f, u, h);
    token_gradients<T, false>(p, s, stash, gate, u, decay, c, P);
  }
  if (PRECISE && s.w == 0 && s.here && p.dh0 && s.chunk == 0)
#pragma unroll
    for (int k = 0; k < VEC; ++k) p.dh0[row + k] = c[k];
  if (p.part) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) back[s.w][slot + k] = P[k];
    lds_barrier();
    if (s.w == 0 && s.here)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float t = 0.0f;
#pragma unroll
        for (int q = 0; q < W; ++q) t += back[q][slot + k];
        p.part[((int64_t)s.chunk * p.batch + s.b) * p.dim + s.c + k] = t;
      }
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
    for (; r + 112 < rows; r += 128) {
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = part[(r + 16 * q) * dim + c];
#pragma unroll
      for (int q = 0; q < 8; ++q) t += v[q];
    }
    for (; r < rows; r += 16) t += part[r * dim + c];
  }
  sums[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < dim) {
    for (int q = 1; q < 16; ++q) t += sums[q][lane];
    ddecay[c] = rows > 0 ? (float)(t / (double)decay[c]) : 0.0f;
  }
}

// ---- one token ----------------------------------------------------------------

// A thread keeps its channels over the rows it takes.  The factor as what it is less
// than 1, in bf16 calls too (4096 x 5120, bf16: 64.1 us, with a itself 63.9).
template <typename T, int VEC>
__global__ __launch_bounds__(256) void step_kernel(const StepArgs p) {
  constexpr bool PRECISE = sizeof(T) == 4;
  const int c = ((int)blockIdx.x * 256 + (int)threadIdx.x) * VEC;
  if (c >= p.dim) return;
  float d[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) d[k] = sum_unit<PRECISE>(p.decay[c + k]);
  for (int64_t row = blockIdx.y; row < p.batch; row += gridDim.y) {
    const int64_t at = row * p.dim + c;
    float x[VEC], r[VEC], i[VEC], h[VEC];
    load_n<VEC>((const T*)p.x + at, x);
    load_n<VEC>((const T*)p.r + at, r);
    load_n<VEC>((const T*)p.i + at, i);
    load_n<VEC>(p.state + at, h);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const Gate g = gate_of<PRECISE, true>(d[k], r[k]);
      h[k] = advance<true>(g.f, h[k], g.m * sigmoid1<PRECISE>(i[k]) * x[k]);
    }
    store_n<VEC>(p.state + at, h);
    store_n<VEC>((T*)p.y + at, h);
  }
}

// ---- launches -------------------------------------------------------------------

int64_t pieces_of(int64_t L, int64_t n) { return L > 0 ? (L + n - 1) / n : 1; }
int64_t up(int64_t n) { return (n + 255) / 256 * 256; }

// Chunks of a group.  Few rows wait for the chain from group to group (about a
// microsecond a link), many for the words that each block reads.  Forwards and
// backwards of 32768 tokens, bf16, inputs from HBM, groups of 4, 8, 16 and 32:
//   64 channels:   44 + 88, 27 + 53, 21 + 37, 19 + 31 us;
//   256:           50 + 91, 36 + 64, 31 + 52, 34 + 55;
//   512:           60 + 107, 46 + 80, 46 + 76, 51 + 85;
//   1024:          75 + 141, 71 + 131, 73 + 135, 80 + 146;
//   2048:          124 + 242, 126 + 245, 129 + 250, 142 + 275;
//   8 x 2048 x 1536: 50 + 92, 51 + 95, 54 + 99, 53 + 110.
int group_of(int64_t rows) { return rows <= 128 ? 32 : rows <= 512 ? 16 : rows <= 1536 ? 8 : 4; }

struct Layout { int64_t ticket, sums, groups, part, bytes; };
// chunk: tokens of a block
Layout layout(int64_t batch, int64_t L, int64_t dim, int chunk, bool need_part) {
  const int64_t chunks = pieces_of(L, chunk), rows = batch * dim, group = group_of(rows);
  Layout a = {};
  int64_t at = 0;
  if (chunks > 1) {
    a.ticket = at; at += 4 * kLine * kCounters;
    a.sums = at;   at += up(8 * chunks * rows);
    a.groups = at; at += up(8 * ((chunks + group - 1) / group) * rows);
  }
  a.part = at;
  if (need_part) at += up(4 * chunks * rows);
  a.bytes = at;
  return a;
}

void place(Args& p, int vec, int chunk) {
  const Layout a = layout(p.batch, p.L, p.dim, chunk, p.ddecay != nullptr);
  char* const ws = (char*)p.ws;
  p.chunks = (int)pieces_of(p.L, chunk);
  p.kept = (int)pieces_of(p.L, kKeep);
  p.group = group_of(p.batch * p.dim);
  p.tiles = (p.dim + 64 * vec - 1) / (64 * vec);
  p.rows = (uint32_t)(p.batch * p.tiles);
  // A counter gives 85 numbers a microsecond.  Calls of as many blocks as run at a
  // time and a little more (768 of the fp32 forward kernel, 1024 of the bf16 one, 512
  // and 768 of the backward ones) take a counter for each row: all begin at once, and
  // wait for their numbers (3 x 1537 x 1000, fp32, 624 blocks: 27 us, with two
  // counters 29.5, with one 31).  More blocks take two counters, which keep them from
  // loading in step (32768 x 2048, bf16: 123 + 234 us, a counter for each row 135 +
  // 257; 8 x 2048 x 1536: 50 + 92, 50 + 96; fp32 3 x 1537 x 1000 backwards, 1200
  // blocks: 45.6, 45.2).
  const uint32_t most = (int64_t)p.rows * p.chunks <= 1024 ? kCounters : 2;
  // rows of a counter, and as few counters as they need: hardly a block is left over
  const uint32_t each = (p.rows + most - 1) / most;
  p.counters = (p.rows + each - 1) / each;
  p.blocks = p.counters * each * (uint32_t)p.chunks;
  p.tickets = (uint32_t*)(ws + a.ticket);
  p.sums = (uint64_t*)(ws + a.sums);
  p.groups = (uint64_t*)(ws + a.groups);
  p.part = p.ddecay ? (float*)(ws + a.part) : nullptr;
}

hipError_t clear(const Args& p, hipStream_t s) {
  // the words of the chunks and of the groups lie side by side, both rounded up to 256 bytes
  const int64_t n = (int64_t)(p.groups - p.sums) +
                    up(8 * (((int64_t)p.chunks + p.group - 1) / p.group * (p.batch * p.dim))) / 8;
  const int64_t blocks = (n + 511) / 512;
  clear_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(p.tickets, p.counters, p.sums, n);
  return hipGetLastError();
}

template <typename T, int VEC, int TOK, int W, bool MANY, bool BWD>
void start_kernel(const Args& p, hipStream_t s) {
  const Grid g = grid_of(p.blocks, 64 * W);
  const dim3 grid(g.x, g.more), block(64 * W);
  if constexpr (BWD) bwd_kernel<T, VEC, TOK, W, MANY><<<grid, block, 0, s>>>(p);
  else fwd_kernel<T, VEC, TOK, W, MANY><<<grid, block, 0, s>>>(p);
}

// SHORT: for calls of kKeep tokens at most (and only the others take the rest)
template <typename T, int VEC, int TOK, int W, bool BWD, bool SHORT>
hipError_t launch(Args p, hipStream_t s) {
  static_assert(TOK * W % kKeep == 0 && kKeep % TOK == 0, "states are kept by whole waves");
  place(p, VEC, TOK * W);
  if constexpr (!SHORT) {
    if (p.chunks > 1) {
      const hipError_t e = clear(p, s);
      if (e != hipSuccess) return e;
      start_kernel<T, VEC, TOK, W, true, BWD>(p, s);
      return hipGetLastError();
    }
  }
  if constexpr (SHORT || TOK * W > kKeep) start_kernel<T, VEC, TOK, W, false, BWD>(p, s);
  return hipGetLastError();
}

// Two bf16 channels a thread instead of one: half as many lanes for the recurrence,
// and a wave's access of 256 bytes instead of 128.  That pays where rows are no whole
// lines of 128 bytes, so that every access touches one more, where there is work
// for the fewer blocks, and where the last tile does not waste it.  Forwards and
// backwards, inputs from HBM, one channel and two:
//   8 x 2048 x 1536: 51 + 93, 56 + 97 us;   1 x 32768 x 2048: 124 + 236, 133 + 267;
//   8 x 2048 x 1535: 66 + 124, 62 + 116;    32 x 1024 x 711: 63 + 123, 59 + 113;
//   1 x 4096 x 711: 17 + 25, 19 + 31;       1 x 32768 x 257: 39 + 66, 48 + 86.
bool pairs(const Args& p) {
  const int64_t tiled = (p.dim + 127) / 128 * (int64_t)128;
  return p.dim % 64 != 0 && 3 * tiled <= 4 * (int64_t)p.dim && p.batch * p.L * p.dim >= 6 << 20;
}

}  // namespace

bool fits(int64_t batch, int64_t L, int64_t dim) {
  // block numbers are 32-bit, and so are chunk numbers and channels
  const __int128 blocks = (__int128)batch * ((dim + 63) / 64) * pieces_of(L, kKeep);
  return dim <= (1 << 24) && L <= 0x7fffff00 && blocks < 0x7fffffff;
}

size_t workspace_bytes(int64_t batch, int64_t L, int64_t dim, bool backward, bool need_ddecay) {
  // the forward's chunks are longer and need less
  return (size_t)layout(batch, L, dim, kKeep, backward && need_ddecay).bytes;
}

// Up to kKeep tokens: one chunk, and a kernel of few instructions, which are most
// of what such a call waits for (33 tokens of 256 channels: 4.7 us, by the kernel
// for longer rows 8.0; calls of 64 x 64 x 1024, bf16: 13.8 and 16.1).
hipError_t forward(const Args& p, bool f32, hipStream_t s) {
  if (p.L <= kKeep)
    return f32 ? launch<float, 1, 4, 16, false, true>(p, s) : launch<bf16_bits, 1, 4, 16, false, true>(p, s);
  if (f32) return launch<float, 1, 16, 8, false, false>(p, s);
  if (pairs(p)) return launch<bf16_bits, 2, 16, 8, false, false>(p, s);
  return launch<bf16_bits, 1, 16, 8, false, false>(p, s);
}

hipError_t backward(const Args& p, bool f32, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (p.batch == 0) {
  } else if (p.L <= kKeep) {
    e = f32 ? launch<float, 1, 4, 16, true, true>(p, s) : launch<bf16_bits, 1, 4, 16, true, true>(p, s);
  } else if (f32) {
    e = launch<float, 1, 8, 8, true, false>(p, s);
  } else {
    e = pairs(p) ? launch<bf16_bits, 2, 8, 8, true, false>(p, s) : launch<bf16_bits, 1, 8, 8, true, false>(p, s);
  }
  if (e != hipSuccess || !p.ddecay) return e;
  const Layout a = layout(p.batch, p.L, p.dim, kKeep, true);
  const int64_t rows = p.L > 0 ? pieces_of(p.L, kKeep) * p.batch : 0;  // without tokens the gradient is 0
  decay_sum_kernel<<<(p.dim + 63) / 64, 1024, 0, s>>>((const float*)((const char*)p.ws + a.part), p.decay,
                                                      p.ddecay, rows, p.dim);
  return hipGetLastError();
}

template <typename T, int VEC>
void launch_step(const StepArgs& p, hipStream_t s) {
  const unsigned x = (unsigned)((p.dim / VEC + 255) / 256);
  int64_t y = 8192 / x;
  y = y < 1 ? 1 : y < p.batch ? y : p.batch;
  step_kernel<T, VEC><<<dim3(x, (unsigned)y), 256, 0, s>>>(p);
}

hipError_t step(const StepArgs& p, bool f32, hipStream_t s) {
  // 16 bytes an access (8 of bf16) where rows allow it
  const bool four = p.dim % 4 == 0;
  if (f32) four ? launch_step<float, 4>(p, s) : launch_step<float, 1>(p, s);
  else four ? launch_step<bf16_bits, 4>(p, s) : launch_step<bf16_bits, 1>(p, s);
  return hipGetLastError();
}

}  // namespace gated_scan
}  // namespace ssm66
