// linattn_walk.h -- the kernel behind linear attention with a decay for each
// head, forward and backward (instantiated in linattn_bf16.hip and
// linattn_f32.hip).
//
// One head, lam = e^g its decay.  Forwards,
//   S_t = lam S_{t-1} + v_t k_t^T,       o_t = scale S_t q_t          (S: Dv x Dk)
// and backwards, with G_t the gradient of S_t,
//   G_t = scale do_t q_t^T + lam G_{t+1},
//   dq_t = scale S_t^T do_t,  dk_t = G_t^T v_t,  dv_t = G_t k_t.
// All four outputs are one computation, a walk over the tokens that keeps a
// state and multiplies it by a row:
//   out_t[x] = sum_s lam^|t-s| (a_t . b_s) c_s[x]  +  (the state from before)
//
//              a    b    c    direction
//     o        q    k    v    forwards
//     dq       do   v    k    forwards
//     dv       k    q    do   backwards
//     dk       v    do   q    backwards
//
// The walk goes in chunks of 64 tokens.  In a chunk, with the state W (V x K,
// V the width of c, K that of a and b) as it enters,
//   out_t = sum_s lam^|t-s| (a_t . b_s) c_s + lam^j(t) W a_t,
//   W'    = lam^n W + sum_s (lam^i(s) c_s) b_s^T,
// all of them products on the matrix cores (v_mfma_f32_16x16x32_bf16).
//
// The gradient of g is taken in the dq walk (DG), forwards and without
// cancellation: T_t = dS_t/dg = lam (T_{t-1} + S_{t-1}), so
//   dg = sum_t scale do_t^T T_t q_t + <dlast, T_last>;
// T walks beside S, and the chunk's part of it is the same intra-chunk product
// with the weights |t-s| lam^|t-s|.
//
// Precision.  Operands of the matrix cores are bf16.  A value that is not one
// is split into bf16 parts that add up to it (x = hi + mid + lo: 8 bits of the
// significand each), and a product of two split values takes the pairs of
// parts whose sizes matter (hi hi; hi mid, mid hi; hi lo, mid mid, lo hi).
// fp32 tensors travel as three parts.  With bf16 tensors the weighted c of
// the state update has three parts, so the state (an fp32 output) is exact to
// fp32 rounding; the scores and the state that multiplies a_t have one part in
// what is rounded to a bf16 output afterwards (their rounding of 2^-9 adds in
// quadrature to the output's own: 2.0e-3 relative RMS against 1.7e-3), three
// in what leads to g's gradient, which is an fp32 sum.  Everything is
// accumulated in fp32.
#pragma once

#include "linattn_launch.h"
#include "ssm_device.h"

namespace ssm66 {
namespace linattn {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(4))) short i16x4;
typedef __attribute__((ext_vector_type(8))) short i16x8;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kQ = kChunk;  // tokens per chunk: the width of a ballot, which holds its document starts
// Word 3 of a raw buffer resource (no stride, 32-bit data format): reads at or
// past the range in word 2 give 0, so rows past a sequence's end and columns
// past a head's width arrive as zeros, whatever memory holds there.
constexpr int kBufferFlags = 0x00020000;
constexpr uint32_t kOutside = 0x7ffffff0u;  // an offset past every range

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float lo_bf(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_bf(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// NPARTS bf16 parts of two floats each, largest first
template <int NPARTS>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t (&part)[NPARTS]) {
#pragma unroll
  for (int i = 0; i < NPARTS; ++i) {
    part[i] = pack_bf16x2(x0, x1);
    x0 -= lo_bf(part[i]);
    x1 -= hi_bf(part[i]);
  }
}

// Matrix results are read a fixed number of cycles after the instruction, and
// the compiler counts the cycles.  It counts a branch as one of them; with a
// branch between a product and the first read of its result, that read has
// given the value from before (seen in the last row of score tiles, fp32
// form, 64 x 32 tile).  So results pass through here before any branch: the
// empty asm keeps each product ahead of it, the wait covers the 8 cycles that
// a 16x16x32 product needs.
template <int N>
__device__ __forceinline__ void settle(f32x4 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(x[i]));
  asm volatile("s_nop 7\n\ts_nop 3");
}

// sum over the pairs of parts (i, j) with i + j < max(PA, PB): the rest is
// below the last bit kept
template <int PA, int PB>
__device__ __forceinline__ f32x4 mfma_parts(const bf16x8 (&a)[PA], const bf16x8 (&b)[PB], f32x4 c) {
  constexpr int M = PA > PB ? PA : PB;
#pragma unroll
  for (int i = PA - 1; i >= 0; --i)  // small terms first
#pragma unroll
    for (int j = PB - 1; j >= 0; --j)
      if (i + j < M) c = mfma(a[i], b[j], c);
  return c;
}

// b and the state sit in LDS in rows of KP bf16, 16-byte piece c of row r at
// c ^ swz(r): 16-byte reads of one piece over rows r .. r + 15 and transposing
// reads of 32 bytes from each of rows r .. r + 3 both spread over the banks.
template <int KP>
__device__ __forceinline__ constexpr int swz(int r) {
  return (((r << 1) & 6) | ((r >> 2) & 1)) ^ (((r >> 3) & 1) * (KP >= 128 ? 8 : 2));
}
template <int KP>
__device__ __forceinline__ constexpr int sw(int r, int col) {
  return (((col >> 3) ^ swz<KP>(r)) << 3) | (col & 7);
}
// c's rows of VB bf16 are only read by the transposing reads (32 bytes from
// each of four rows at a time): pairs of pieces change places by row
template <int VB>
__device__ __forceinline__ constexpr int swc(int r, int col) {
  constexpr int kShift = VB == 64 ? 0 : 1;
  constexpr int kMask = VB == 64 ? 3 : (VB == 32 ? 1 : 0);
  return (((col >> 3) ^ (((r >> kShift) & kMask) << 1)) << 3) | (col & 7);
}

// Transposing reads: the operand "row l % 16, k = ..." of a matrix stored
// k-major.  Lane i of each 16 receives, as its 4 values, element i % 4 of the
// 8 bytes addressed by lanes 4 k + i / 4, k = 0..3, of its group.
__device__ __forceinline__ i16x4 tr_read(const __bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(void*)p);
}
__device__ __forceinline__ bf16x8 join(i16x4 a, i16x4 b) {
  const i16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}

template <int NP>
struct Io { typedef bf16_bits T; };
template <>
struct Io<3> { typedef float T; };

template <int NP, int KP, int VB, bool DG, bool STATE>
struct Shape {
  static constexpr int PS = STATE ? 0 : (NP == 3 || DG ? 3 : 1);            // parts of the state
  // the fp32 form with 256-wide rows keeps two parts of T: three do not fit the LDS
  static constexpr int PT = (STATE || !DG) ? 0 : (NP == 3 && KP == 256 ? 2 : 3);
  static constexpr int PW = 3;                                             // parts of the weighted c
  static constexpr int NC = STATE ? 0 : NP;
  static constexpr int NW2 = DG ? PW : 0;
  static constexpr int kB = NP * kQ * KP;
  static constexpr int kC = NC * kQ * VB;
  static constexpr int kW = PW * kQ * VB;
  static constexpr int kW2 = NW2 * kQ * VB;
  static constexpr int kS = PS * VB * KP;
  static constexpr int kT = PT * VB * KP;
  static constexpr int kElems = kB + kC + kW + kW2 + kS + kT;
  static constexpr bool kFits = 2 * kElems + 1024 <= 160 * 1024;  // the LDS of a CU
};

__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// lam^e for e >= 0 (1 at e = 0 also where lam is 0)
__device__ __forceinline__ float power(float g2, int e) {
  return e == 0 ? 1.0f : exp2_hw(g2 * (float)e);
}

template <int NP, int KP, int VB, bool REV, bool DG, bool STATE>
__global__ __launch_bounds__(256, NP == 1 ? 2 : 1) void walk_kernel(const WalkArgs p) {
  typedef typename Io<NP>::T T;
  typedef Shape<NP, KP, VB, DG, STATE> Sh;
  constexpr int ES = sizeof(T);
  constexpr int EPP = 16 / ES;                 // elements of a 16-byte piece
  constexpr int PRB = KP / EPP;                // pieces in a row of b
  constexpr int PRC = VB / EPP;                // pieces in a row of c
  constexpr int RB = kQ * PRB / 256;           // pieces of b per thread
  constexpr int RC = kQ * PRC / 256;
  constexpr int NK = KP / 32;                  // k-steps of a . b
  constexpr int NV = VB / 16;                  // column tiles of out
  constexpr int JK = KP / 64;                  // row tiles of the state per wave
  constexpr int RA = NP == 1 ? NK : 2 * NK;    // 16-byte pieces of a per lane
  static_assert(RB >= 1 && RC >= 1 && JK >= 1, "tile too small");

  __shared__ __align__(16) __bf16 lds[Sh::kElems];
  __bf16* const Bs = lds;
  __bf16* const Cs = Bs + Sh::kB;
  __bf16* const Cw = Cs + Sh::kC;
  __bf16* const Cw2 = Cw + Sh::kW;
  __bf16* const Ss = Cw2 + Sh::kW2;
  __bf16* const Ts = Ss + Sh::kS;

  // Consecutive block ids go round-robin to the 8 XCDs; each XCD gets a
  // contiguous run of (entry, head, span, slice), so the slices that read the
  // same a and b meet in its L2.
  const uint32_t per = (p.nblk + 7u) / 8u;
  const uint32_t logical = (blockIdx.x % 8u) * per + blockIdx.x / 8u;
  if (logical >= p.nblk) return;
  uint32_t rest = logical;
  const int sl = (int)(rest % (uint32_t)p.nsl);
  rest /= (uint32_t)p.nsl;
  const int span = (int)(rest % (uint32_t)p.nspan_run);
  rest /= (uint32_t)p.nspan_run;
  const int h = (int)(rest % (uint32_t)p.H);
  const int b = (int)(rest / (uint32_t)p.H);

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = lane >> 4;
  const int K = p.K, V = p.V;
  const int v0 = sl * VB;
  const float g2 = p.log_decay[h] * kLog2e;
  const float lam64 = power(g2, kQ);

  const int64_t L = p.L;
  int64_t len = L;
  if (p.seq_lens) {
    const int64_t n = p.seq_lens[b];
    len = n < 0 ? 0 : (n < L ? n : L);
  }
  const int nc = (int)((L + kQ - 1) / kQ);        // chunks of the tensor
  const int nlive = (int)((len + kQ - 1) / kQ);   // chunks that hold real tokens
  auto chunk_of = [&](int i) { return REV ? nc - 1 - i : i; };  // i-th chunk of the walk
  auto live_in = [&](int c) {
    const int64_t n = len - (int64_t)c * kQ;
    return n <= 0 ? 0 : (n < kQ ? (int)n : kQ);
  };
  const int i0 = span * p.span_chunks;
  const int i1 = i0 + p.span_chunks < nc ? i0 + p.span_chunks : nc;

  // ---- where this block's rows are.  One sequence and head of a tensor of
  // (L, heads, width): byte offsets within a chunk fit 32 bits (the launch
  // bounds heads * width).
  const int64_t bL = (int64_t)b * L;
  const uint32_t rsa = (uint32_t)p.Ha * K * ES, rsb = (uint32_t)p.Hb * K * ES, rsc = (uint32_t)p.Hc * V * ES;
  const char* const pa = STATE ? nullptr : (const char*)p.a + (bL * p.Ha + h / (p.H / p.Ha)) * (int64_t)K * ES;
  const char* const pb = (const char*)p.b + (bL * p.Hb + h / (p.H / p.Hb)) * (int64_t)K * ES;
  const char* const pc = (const char*)p.c + ((bL * p.Hc + h / (p.H / p.Hc)) * (int64_t)V + v0) * ES;
  const char* const px = DG && !STATE ? (const char*)p.x + ((bL * p.Hc + h / (p.H / p.Hc)) * (int64_t)V + v0) * ES : nullptr;

  u32x4 rB[RB], rC[RC], rA[STATE ? 1 : RA];
  uint32_t rR = 0;
  const int rowB = tid / PRB, pieceB = tid % PRB;
  const int rowC = tid / PRC, pieceC = tid % PRC;
  auto load_chunk = [&](int c) {
    const int n = live_in(c);
    const int64_t t0 = (int64_t)c * kQ;
    {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(pb + t0 * rsb), (short)0, n ? (int)((uint32_t)(n - 1) * rsb + (uint32_t)K * ES) : 0, kBufferFlags);
      const uint32_t o = pieceB * EPP < K ? (uint32_t)rowB * rsb + pieceB * 16u : kOutside;
#pragma unroll
      for (int j = 0; j < RB; ++j)
        rB[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            r, (int)(o == kOutside ? o : o + (uint32_t)j * (256u / PRB) * rsb), 0, 0));
    }
    {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(pc + t0 * rsc), (short)0, n ? (int)((uint32_t)(n - 1) * rsc + (uint32_t)(V - v0) * ES) : 0, kBufferFlags);
      const uint32_t o = v0 + pieceC * EPP < V ? (uint32_t)rowC * rsc + pieceC * 16u : kOutside;
#pragma unroll
      for (int j = 0; j < RC; ++j)
        rC[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            r, (int)(o == kOutside ? o : o + (uint32_t)j * (256u / PRC) * rsc), 0, 0));
    }
    if constexpr (!STATE) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(pa + t0 * rsa), (short)0, n ? (int)((uint32_t)(n - 1) * rsa + (uint32_t)K * ES) : 0, kBufferFlags);
      const uint32_t o = (uint32_t)(16 * w + lr) * rsa + (uint32_t)lk * 8u * ES;
#pragma unroll
      for (int j = 0; j < RA; ++j) {
        const int k = NP == 1 ? j : j / 2, half = NP == 1 ? 0 : j % 2;
        const bool in = 32 * k + 8 * lk < K;
        rA[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            r, (int)(in ? o + (uint32_t)(32 * k * ES + 16 * half) : kOutside), 0, 0));
      }
    }
    if (p.reset) {
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)(p.reset + bL + t0), (short)0, n, kBufferFlags);
      rR = __builtin_amdgcn_raw_buffer_load_b8(r, lane, 0, 0);
    }
  };

  // ---- a chunk from the registers into LDS
  bf16x8 aF[STATE ? 1 : NK][NP];
  uint64_t starts = 0;  // document starts of the staged chunk, one bit per token
  auto stage = [&](int n) {
    starts = p.reset ? __ballot((rR & 0xffu) != 0) : 0;
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int row = rowB + j * (256 / PRB), col = pieceB * EPP;
      __bf16* d = Bs + row * KP + sw<KP>(row, col);
      if constexpr (NP == 1) {
        *(u32x4*)d = rB[j];
      } else {
        uint32_t p0[3], p1[3];
        split2<3>(__uint_as_float(rB[j][0]), __uint_as_float(rB[j][1]), p0);
        split2<3>(__uint_as_float(rB[j][2]), __uint_as_float(rB[j][3]), p1);
#pragma unroll
        for (int q = 0; q < 3; ++q) *(u32x2*)(d + q * kQ * KP) = u32x2{p0[q], p1[q]};
      }
    }
#pragma unroll
    for (int j = 0; j < RC; ++j) {
      const int row = rowC + j * (256 / PRC), col = pieceC * EPP;
      const int at = row * VB + swc<VB>(row, col);
      // the weight of this token in the state at the walk's end of the chunk
      const int e = REV ? row + 1 : n - 1 - row;
      const bool reaches = REV ? (starts & low_bits(row + 1)) == 0 : ((starts >> row) >> 1) == 0;
      const bool in = row < n && reaches;
      const float wt = in ? p.s_state * power(g2, e) : 0.0f;
      float f[EPP];
#pragma unroll
      for (int i = 0; i < EPP; ++i)
        f[i] = NP == 1 ? ((i & 1) ? hi_bf(rC[j][i / 2]) : lo_bf(rC[j][i / 2])) : __uint_as_float(rC[j][i % 4]);
      if constexpr (!STATE) {
        if constexpr (NP == 1) {
          *(u32x4*)(Cs + at) = rC[j];
        } else {
          uint32_t p0[3], p1[3];
          split2<3>(f[0], f[1], p0);
          split2<3>(f[2], f[3], p1);
#pragma unroll
          for (int q = 0; q < 3; ++q) *(u32x2*)(Cs + q * kQ * VB + at) = u32x2{p0[q], p1[q]};
        }
      }
#pragma unroll
      for (int which = 0; which < (DG ? 2 : 1); ++which) {
        const float wq = which == 0 ? wt : wt * (float)(in ? e : 0);
        __bf16* const d = (which == 0 ? Cw : Cw2) + at;
        uint32_t pt[EPP / 2][3];
#pragma unroll
        for (int i = 0; i < EPP / 2; ++i) {
          const float x0 = in ? f[2 * i] * wq : 0.0f, x1 = in ? f[2 * i + 1] * wq : 0.0f;
          split2<3>(x0, x1, pt[i]);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          if constexpr (NP == 1)
            *(u32x4*)(d + q * kQ * VB) = u32x4{pt[0][q], pt[1][q], pt[EPP / 2 - 2][q], pt[EPP / 2 - 1][q]};
          else
            *(u32x2*)(d + q * kQ * VB) = u32x2{pt[0][q], pt[1][q]};
        }
      }
    }
    if constexpr (!STATE) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        if constexpr (NP == 1) {
          aF[k][0] = __builtin_bit_cast(bf16x8, rA[k]);
        } else {
          uint32_t pt[4][3];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            split2<3>(__uint_as_float(rA[2 * k + i / 2][2 * (i % 2)]),
                      __uint_as_float(rA[2 * k + i / 2][2 * (i % 2) + 1]), pt[i]);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            aF[k][q] = __builtin_bit_cast(bf16x8, u32x4{pt[0][q], pt[1][q], pt[2][q], pt[3][q]});
        }
      }
    }
  };

  // ---- the state, fp32, in the matrix cores' result layout: wave w holds
  // row tiles kt = w + 4 j; lane value i is W[v = 16 vt + lr][kappa = 16 kt + 4 lk + i]
  f32x4 S[JK][NV], D[DG ? JK : 1][DG ? NV : 1];
  const int64_t bh = (int64_t)b * p.H + h;
  const int64_t state_elems = (int64_t)K * V;
#pragma unroll
  for (int j = 0; j < JK; ++j)
#pragma unroll
    for (int vt = 0; vt < NV; ++vt) {
      S[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (DG) D[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  if constexpr (!STATE) {
    auto for_state = [&](auto&& f) {
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NV; ++vt) {
          const int v = v0 + 16 * vt + lr, k = 16 * (w + 4 * j) + 4 * lk;
          if (v < V && k < K) f(j, vt, v, k);
        }
    };
    if (p.init) {
      const float* s0 = p.init + bh * state_elems;
      for_state([&](int j, int vt, int v, int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][vt][i] = s0[v * p.state_sv + (k + i) * p.state_sk];
      });
    }
    // the states that the spans before this one add, in the walk's order
    for (int m = 0; m < span; ++m) {
      const float* loc = p.ws + ((int64_t)m * p.batch * p.H + bh) * (DG ? 2 : 1) * state_elems;
      // real tokens of the span
      const int m0 = m * p.span_chunks, m1 = m0 + p.span_chunks - 1;
      const int64_t ca = chunk_of(REV ? m1 : m0), cb = chunk_of(REV ? m0 : m1) + 1;
      int64_t hi = cb * kQ < len ? cb * kQ : len;
      const int64_t n = hi > ca * kQ ? hi - ca * kQ : 0;
      const bool cut = p.span_cut[(int64_t)m * p.batch + b] != 0;
      const float d = n == 0 ? 1.0f : (cut ? 0.0f : exp2_hw(g2 * (float)n));
      for_state([&](int j, int vt, int v, int k) {
        const float4 a = *(const float4*)(loc + (int64_t)v * K + k);
        const float av[4] = {a.x, a.y, a.z, a.w};
        if constexpr (DG) {
          const float4 t = *(const float4*)(loc + state_elems + (int64_t)v * K + k);
          const float tv[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            D[j][vt][i] = cut ? tv[i] : d * (D[j][vt][i] + (float)n * S[j][vt][i]) + tv[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][vt][i] = cut ? av[i] : d * S[j][vt][i] + av[i];
      });
    }
  }
  // the state's parts into LDS: four consecutive kappa of one row per lane
  auto put_state = [&]() {
    if constexpr (!STATE) {
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NV; ++vt) {
          const int at = (16 * vt + lr) * KP + sw<KP>(lr, 16 * (w + 4 * j) + 4 * lk);
          {
            uint32_t p0[Sh::PS], p1[Sh::PS];
            split2<Sh::PS>(S[j][vt][0], S[j][vt][1], p0);
            split2<Sh::PS>(S[j][vt][2], S[j][vt][3], p1);
#pragma unroll
            for (int q = 0; q < Sh::PS; ++q) *(u32x2*)(Ss + q * VB * KP + at) = u32x2{p0[q], p1[q]};
          }
          if constexpr (DG) {
            uint32_t p0[Sh::PT], p1[Sh::PT];
            split2<Sh::PT>(D[j][vt][0], D[j][vt][1], p0);
            split2<Sh::PT>(D[j][vt][2], D[j][vt][3], p1);
#pragma unroll
            for (int q = 0; q < Sh::PT; ++q) *(u32x2*)(Ts + q * VB * KP + at) = u32x2{p0[q], p1[q]};
          }
        }
    }
  };

  // ---- lane constants of the intra-chunk weights, of token t = 16 W + lr and
  // s = 16 sb + 4 lk + i: on the diagonal block lam^|lr - 4 lk - i|, m blocks
  // away lam^(16 m - 16) times the weight one block away
  float wd[4], w1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = REV ? 4 * lk + i - lr : lr - 4 * lk - i;  // tokens from s to t along the walk
    wd[i] = e >= 0 ? power(g2, e) : 0.0f;
    w1[i] = power(g2, 16 + e);  // e > -16
  }
  const float lam16 = power(g2, 16);
  float dg = 0.0f;

  // ---- the outputs of token block W (uniform in a wave) of the staged chunk
  auto outputs = [&](auto Wc, int c, int n) {
    constexpr int W = decltype(Wc)::value;
    constexpr int PP = NP == 3 ? 3 : 1;  // parts of the scores that lead to out
    const int t = 16 * W + lr;
    const int64_t row = bL + (int64_t)c * kQ + t;
    // x of this lane's outputs, asked for early
    u32x4 rX[DG ? NV : 1];
    if constexpr (DG) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(px + (int64_t)c * kQ * rsc), (short)0, (int)((uint32_t)(n - 1) * rsc + (uint32_t)(V - v0) * ES), kBufferFlags);
#pragma unroll
      for (int vt = 0; vt < NV; ++vt) {
        const int col = 16 * vt + 4 * lk;
        const int o = (int)(v0 + col < V ? (uint32_t)t * rsc + (uint32_t)col * ES : kOutside);
        if constexpr (NP == 1) {
          const u32x2 q = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, o, 0, 0));
          rX[vt] = u32x4{q[0] << 16, q[0] & 0xffff0000u, q[1] << 16, q[1] & 0xffff0000u};
        } else {
          rX[vt] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0));
        }
      }
    }
    // the state's part: acc = W a_t (rows v, columns t)
    f32x4 acc[NV], acc2[DG ? NV : 1];
    const int je = REV ? n - 1 - t : t + 1;
    const bool sees = REV ? ((starts >> t) >> 1) == 0 : (starts & low_bits(t + 1)) == 0;
    const bool from = sees && t < n;
    const float wi = from ? p.s_inter * power(g2, je > 0 ? je : 0) : 0.0f;
#pragma unroll
    for (int vt = 0; vt < NV; ++vt) {
      f32x4 q = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        bf16x8 sF[Sh::PS > 0 ? Sh::PS : 1];
#pragma unroll
        for (int e = 0; e < Sh::PS; ++e)
          sF[e] = *(const bf16x8*)(Ss + e * VB * KP + (16 * vt + lr) * KP + sw<KP>(lr, 32 * k + 8 * lk));
        q = mfma_parts(sF, aF[k], q);
      }
      if constexpr (DG) {
        f32x4 u = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          bf16x8 sF[Sh::PT > 0 ? Sh::PT : 1];
#pragma unroll
          for (int e = 0; e < Sh::PT; ++e)
            sF[e] = *(const bf16x8*)(Ts + e * VB * KP + (16 * vt + lr) * KP + sw<KP>(lr, 32 * k + 8 * lk));
          u = mfma_parts(sF, aF[k], u);
        }
        acc2[vt] = u;
      }
      acc[vt] = q;
    }
    settle(acc);
    if constexpr (DG) settle(acc2);
#pragma unroll
    for (int vt = 0; vt < NV; ++vt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DG) acc2[vt][i] = from ? wi * (acc2[vt][i] + (float)je * acc[vt][i]) : 0.0f;
        acc[vt][i] = from ? wi * acc[vt][i] : 0.0f;
      }
    // the chunk's own part, two 16-token blocks of s at a time: scores
    // transposed (s by t), weighted, and as they stand the operand of the
    // product with c
#pragma unroll
    for (int pair = REV ? W / 2 : 0; pair <= (REV ? 1 : W / 2); ++pair) {
      uint32_t pw[2][2][PP], pw2[2][2][DG ? 3 : 1];  // [block][half][part]
      f32x4 g[2];
      uint32_t sees_s[2];  // bit i: token t sees token s = 16 sb + 4 lk + i
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int sb = 2 * pair + u;
        const int m = REV ? sb - W : W - sb;  // blocks from s to t
        g[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        sees_s[u] = 0;
        if (m < 0) continue;
        sees_s[u] = m > 0 ? 15u : 0u;
        if (m == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sees_s[u] |= (REV ? 4 * lk + i >= lr : 4 * lk + i <= lr) ? 1u << i : 0u;
        }
        if (starts) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int s = 16 * sb + 4 * lk + i;
            const int lo = REV ? t : s, hi = REV ? s : t;
            if ((starts & low_bits(hi + 1) & ~low_bits(lo + 1)) != 0) sees_s[u] &= ~(1u << i);
          }
        }
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          bf16x8 bF[NP];
#pragma unroll
          for (int e = 0; e < NP; ++e)
            bF[e] = *(const bf16x8*)(Bs + e * kQ * KP + (16 * sb + lr) * KP + sw<KP>(lr, 32 * k + 8 * lk));
          g[u] = mfma_parts(bF, aF[k], g[u]);
        }
      }
      settle(g);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int sb = 2 * pair + u;
        const int m = REV ? sb - W : W - sb;
        const float f = m >= 3 ? p.s_intra * lam16 * lam16 : (m == 2 ? p.s_intra * lam16 : p.s_intra);
        float x[4], x2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = g[u][i] * (f * (m <= 0 ? wd[i] : w1[i]));
          x[i] = (sees_s[u] >> i) & 1u ? y : 0.0f;
          if constexpr (DG) x2[i] = x[i] * (float)(16 * m + (REV ? 4 * lk + i - lr : lr - 4 * lk - i));
        }
        split2<PP>(x[0], x[1], pw[u][0]);
        split2<PP>(x[2], x[3], pw[u][1]);
        if constexpr (DG) {
          split2<3>(x2[0], x2[1], pw2[u][0]);
          split2<3>(x2[2], x2[3], pw2[u][1]);
        }
      }
      bf16x8 pF[PP], pF2[DG ? 3 : 1];
#pragma unroll
      for (int e = 0; e < PP; ++e)
        pF[e] = __builtin_bit_cast(bf16x8, u32x4{pw[0][0][e], pw[0][1][e], pw[1][0][e], pw[1][1][e]});
      if constexpr (DG) {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          pF2[e] = __builtin_bit_cast(bf16x8, u32x4{pw2[0][0][e], pw2[0][1][e], pw2[1][0][e], pw2[1][1][e]});
      }
      const int g4 = lane >> 4, kk = (lane & 15) >> 2, qq = lane & 3;
      const int ra = 32 * pair + 4 * g4 + kk, rb = ra + 16;
#pragma unroll
      for (int vt = 0; vt < NV; ++vt) {
        bf16x8 cF[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e)
          cF[e] = join(tr_read(Cs + e * kQ * VB + ra * VB + swc<VB>(ra, 16 * vt + 4 * qq)),
                       tr_read(Cs + e * kQ * VB + rb * VB + swc<VB>(rb, 16 * vt + 4 * qq)));
        acc[vt] = mfma_parts(cF, pF, acc[vt]);
        if constexpr (DG) acc2[vt] = mfma_parts(cF, pF2, acc2[vt]);
      }
    }
    settle(acc);
    if constexpr (DG) settle(acc2);
    // out rows of real tokens, and zeros at padding inside the chunk
    if (row < bL + L) {
#pragma unroll
      for (int vt = 0; vt < NV; ++vt) {
        const int v = v0 + 16 * vt + 4 * lk;
        if (v < V) {
          const f32x4 o = t < n ? acc[vt] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          const int64_t at = (row * p.H + h) * V + v;
          if (NP == 3 || p.out_f32)
            *(float4*)((float*)p.out + at) = float4{o[0], o[1], o[2], o[3]};
          else
            *(u32x2*)((bf16_bits*)p.out + at) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        }
      }
    }
    if constexpr (DG) {
#pragma unroll
      for (int vt = 0; vt < NV; ++vt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t < n) dg = fmaf(acc2[vt][i], __uint_as_float(rX[vt][i]), dg);
    }
  };

  // ---- the state at the walk's end of the staged chunk
  auto update = [&](int n) {
    const bool cut = starts != 0;
    const float d = cut ? 0.0f : (n == kQ ? lam64 : power(g2, n));
    const float nf = (float)n;
#pragma unroll
    for (int j = 0; j < JK; ++j)
#pragma unroll
      for (int vt = 0; vt < NV; ++vt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DG) D[j][vt][i] = cut ? 0.0f : d * (D[j][vt][i] + nf * S[j][vt][i]);
          S[j][vt][i] = cut ? 0.0f : d * S[j][vt][i];
        }
    const int g4 = lane >> 4, kk = (lane & 15) >> 2, qq = lane & 3;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int ra = 32 * ks + 8 * g4 + kk, rb = ra + 4;
      bf16x8 bF[JK][NP];
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const int col = 16 * (w + 4 * j) + 4 * qq;
          bF[j][e] = join(tr_read(Bs + e * kQ * KP + ra * KP + sw<KP>(ra, col)),
                          tr_read(Bs + e * kQ * KP + rb * KP + sw<KP>(rb, col)));
        }
#pragma unroll
      for (int vt = 0; vt < NV; ++vt) {
        const int col = 16 * vt + 4 * qq;
        bf16x8 cF[3];
#pragma unroll
        for (int e = 0; e < 3; ++e)
          cF[e] = join(tr_read(Cw + e * kQ * VB + ra * VB + swc<VB>(ra, col)),
                       tr_read(Cw + e * kQ * VB + rb * VB + swc<VB>(rb, col)));
#pragma unroll
        for (int j = 0; j < JK; ++j) S[j][vt] = mfma_parts(bF[j], cF, S[j][vt]);
        if constexpr (DG) {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            cF[e] = join(tr_read(Cw2 + e * kQ * VB + ra * VB + swc<VB>(ra, col)),
                         tr_read(Cw2 + e * kQ * VB + rb * VB + swc<VB>(rb, col)));
#pragma unroll
          for (int j = 0; j < JK; ++j) D[j][vt] = mfma_parts(bF[j], cF, D[j][vt]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < JK; ++j) {
      settle(S[j]);
      if constexpr (DG) settle(D[j]);
    }
  };

  // ---- the walk
  const int first = REV ? (i0 > nc - nlive ? i0 : nc - nlive) : i0;
  const int last = REV ? i1 : (i1 < nlive ? i1 : nlive);
  int any_start = 0;
  if (first < last) {
    load_chunk(chunk_of(first));
    stage(live_in(chunk_of(first)));
    put_state();
    lds_barrier();
    for (int i = first; i < last; ++i) {
      const int c = chunk_of(i), n = live_in(c);
      if (i + 1 < last) load_chunk(chunk_of(i + 1));
      if constexpr (!STATE) {
        if (w == 0) outputs(std::integral_constant<int, 0>{}, c, n);
        else if (w == 1) outputs(std::integral_constant<int, 1>{}, c, n);
        else if (w == 2) outputs(std::integral_constant<int, 2>{}, c, n);
        else outputs(std::integral_constant<int, 3>{}, c, n);
      }
      any_start |= starts != 0;
      update(n);
      if (i + 1 < last) {
        lds_barrier();
        stage(live_in(chunk_of(i + 1)));
        put_state();
        lds_barrier();
      }
    }
  }

  if constexpr (STATE) {
    float* loc = p.ws + ((int64_t)span * p.batch * p.H + bh) * (DG ? 2 : 1) * state_elems;
#pragma unroll
    for (int j = 0; j < JK; ++j)
#pragma unroll
      for (int vt = 0; vt < NV; ++vt) {
        const int v = v0 + 16 * vt + lr, k = 16 * (w + 4 * j) + 4 * lk;
        if (v < V && k < K) {
          *(f32x4*)(loc + (int64_t)v * K + k) = S[j][vt];
          if constexpr (DG) *(f32x4*)(loc + state_elems + (int64_t)v * K + k) = D[j][vt];
        }
      }
    if (h == 0 && sl == 0 && tid == 0) p.span_cut[(int64_t)span * p.batch + b] = any_start;
  } else {
    // padding rows of the span that no chunk above held: zeros
    const int ca = chunk_of(REV ? i1 - 1 : i0), cb = chunk_of(REV ? i0 : i1 - 1) + 1;
    const int64_t z0 = ((int64_t)(ca > nlive ? ca : nlive)) * kQ;
    const int64_t z1 = (int64_t)cb * kQ < L ? (int64_t)cb * kQ : L;
    const int cols = V - v0 < VB ? V - v0 : VB;
    for (int64_t q = tid; q < (z1 - z0) * (VB / 4); q += 256) {
      const int64_t row = bL + z0 + q / (VB / 4);
      const int v = 4 * (int)(q % (VB / 4));
      if (v < cols) {
        const int64_t at = (row * p.H + h) * V + v0 + v;
        if (NP == 3 || p.out_f32)
          *(float4*)((float*)p.out + at) = float4{0.0f, 0.0f, 0.0f, 0.0f};
        else
          *(u32x2*)((bf16_bits*)p.out + at) = u32x2{0u, 0u};
      }
    }
    const bool ends = span == p.nspan - 1;  // this block ends the walk
    if (ends && p.final_state) {
      float* fs = p.final_state + bh * state_elems;
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NV; ++vt) {
          const int v = v0 + 16 * vt + lr, k = 16 * (w + 4 * j) + 4 * lk;
          if (v < V && k < K) *(f32x4*)(fs + (int64_t)v * K + k) = S[j][vt];
        }
    }
    if constexpr (DG) {
      if (ends && p.dlast) {  // <dlast, T after the last token>; dlast is K-major here
        const float* dl = p.dlast + bh * state_elems;
#pragma unroll
        for (int j = 0; j < JK; ++j)
#pragma unroll
          for (int vt = 0; vt < NV; ++vt) {
            const int v = v0 + 16 * vt + lr, k = 16 * (w + 4 * j) + 4 * lk;
            if (v < V && k < K) {
#pragma unroll
              for (int i = 0; i < 4; ++i) dg = fmaf(dl[(int64_t)(k + i) * V + v], D[j][vt][i], dg);
            }
          }
      }
      // the block's sum, in a fixed order
      __shared__ float sums[256];
      sums[tid] = dg;
      __syncthreads();
#pragma unroll
      for (int s = 128; s > 0; s >>= 1) {
        if (tid < s) sums[tid] += sums[tid + s];
        __syncthreads();
      }
      if (tid == 0)
        p.dg_part[(int64_t)h * p.batch * p.nsl * p.nspan + ((int64_t)b * p.nsl + sl) * p.nspan + span] = sums[0];
    }
  }
}

template <int NP, int KP, int VB>
hipError_t launch_walk(const WalkArgs& args, bool rev, bool dg, bool state, hipStream_t stream) {
  WalkArgs a = args;
  a.nspan_run = state ? a.nspan - 1 : a.nspan;
  a.nsl = (a.V + VB - 1) / VB;
  const int64_t n = (int64_t)a.batch * a.H * a.nsl * a.nspan_run;
  if (n == 0) return hipSuccess;
  a.nblk = (uint32_t)n;
  const dim3 grid((uint32_t)((n + 7) / 8 * 8));
  if (state) {
    if (rev) walk_kernel<NP, KP, VB, true, false, true><<<grid, 256, 0, stream>>>(a);
    else if (dg) walk_kernel<NP, KP, VB, false, true, true><<<grid, 256, 0, stream>>>(a);
    else walk_kernel<NP, KP, VB, false, false, true><<<grid, 256, 0, stream>>>(a);
  } else {
    if (rev) walk_kernel<NP, KP, VB, true, false, false><<<grid, 256, 0, stream>>>(a);
    else if (dg) {
      if constexpr (Shape<NP, KP, VB, true, false>::kFits)
        walk_kernel<NP, KP, VB, false, true, false><<<grid, 256, 0, stream>>>(a);
      else
        return hipErrorInvalidValue;  // walk_tile takes a narrower tile
    }
    else walk_kernel<NP, KP, VB, false, false, false><<<grid, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace linattn
}  // namespace ssm66
