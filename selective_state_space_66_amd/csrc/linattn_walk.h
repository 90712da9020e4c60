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
// fp32 rounding.  Where they lead to a bf16 output, the scores and the state
// that multiplies a_t have two parts: 2^-18 of a value is left out, and the
// output's error is that of its one rounding to four digits (8 x 2048 tokens of
// 24 heads, 128 keys, 64 values: 1.6586e-3 relative RMS, as the exact result's
// rounding; with one part of the state 2.2859e-3 and 75 us for 82, with three
// parts of both 96 us).  Where they lead to g's gradient, an fp32 sum, both have
// three.  Everything is accumulated in fp32.
//
// Work split.  A block owns one entry, head, span of the tokens and VB columns
// of c.  A chunk's steps form a chain (state, outputs, next state), and with
// one wave of a block per SIMD its latencies add up, so a block has two groups
// of four or eight waves that work on a chunk at the same time.  Group A makes
// the outputs, with the rows of a straight from memory in operand registers.
// Group B keeps the state in registers, updates it, and brings b and c in: it
// stages chunk i + 1 while chunk i is worked on, from loads issued a chunk
// earlier, into the other of two buffers: one barrier per chunk.  Where the LDS
// does not hold two of everything, the rows of b and c have two and the
// weighted c and the state one, written after a second barrier behind their
// readers; or everything has one.  fp32 rows of 256 with the log-decay's
// gradient fill the LDS even so: there c lies where T's last part was, brought
// in between two barriers of its own once group A has read T.
// Chunks of 64 tokens: the starts of documents fit one ballot.
//
// What bounds it.  About 60 flops per byte of bf16 rows: at the rates of a
// large copy and a large product the bytes take longer.  8 x 2048 tokens of 24
// heads, 128 keys and 64 values, bf16: 77 to 86 us (3.6 to 4.0 TB/s; a copy of
// these bytes takes 59), a third of the matrix cycles used.  The other walks are
// bound by the latency of a chunk's chain: with the log-decay's gradient 230 to
// 255 us at the same size (19% of the matrix cycles, 38% of the vector ones and
// 45% of the LDS's are used; without group A's products 180, without B's 237,
// without both 97), fp32 rows of 72 and 96 with 3 x 1537 tokens of 12 heads 54.
#pragma once

#include "linattn_launch.h"
#include "lm_grid.h"
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
// Cache policy of the output's stores: non-temporal.  The loads and stores of a
// walk without its arithmetic took 52 us this way and 72 us with plain stores
// (8 x 2048 x 24 heads, 128 keys, 64 values); nt loads gained nothing.
constexpr int kNt = 2;
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
// c ^ swz(r), for 16-byte reads of one piece over rows r .. r + 15 and
// transposing reads of 32 bytes from each of rows r .. r + 3.  Rows of 96 need
// no exchange, 52 banks apart.
template <int KP>
constexpr int kRow = KP == 96 ? 104 : KP;
template <int KP>
__device__ __forceinline__ constexpr int swz(int r) {
  return (((r << 1) & 6) | ((r >> 2) & 1)) ^ (((r >> 3) & 1) * (KP >= 128 ? 8 : 2));
}
template <int KP>
__device__ __forceinline__ constexpr int sw(int r, int col) {
  return KP == 96 ? col : (((col >> 3) ^ swz<KP>(r)) << 3) | (col & 7);
}
// c's rows of VB bf16 are only read by the transposing reads (32 bytes from
// each of four rows at a time, over 64 banks of 4 bytes): where one row or two
// fill the banks, the others change places by pairs of pieces.  Rows of 32 stay
// as they are, and a read of theirs meets half of the banks: of the LDS's active
// cycles 41% are conflicts in a walk of 32 columns, 43% with the log-decay's
// gradient, 26% in one of 64 columns.
template <int VB>
__device__ __forceinline__ constexpr int swc(int r, int col) {
  return VB >= 64 ? (((col >> 3) ^ ((VB == 128 ? r & 3 : (r >> 1) & 1) << 1)) << 3) | (col & 7) : col;
}

// The contractions over kappa take it in steps of 32; lane group lk of step k
// holds the 8 values from here on (any split that both operands share gives
// the same sums; this one is what the loads of a deliver)
template <int NP>
__device__ __forceinline__ constexpr int kcol(int k, int lk) {
  return NP == 1 ? 64 * (k / 2) + 16 * lk + 8 * (k % 2) : 32 * k + 8 * lk;
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
  static constexpr int PS = STATE ? 0 : (NP == 3 || DG ? 3 : 2);  // parts of the state
  static constexpr int PT = (STATE || !DG) ? 0 : 3;
  static constexpr int PW = 3;                                    // parts of the weighted c
  static constexpr int KS = kRow<KP>;
  static constexpr int kB = NP * kQ * KS;                         // one buffer of b
  // c in the place of T's last part: with one of its own this shape takes 162 KB
  static constexpr bool kShared = NP == 3 && KP == 256 && DG && !STATE;
  static constexpr int kC = STATE || kShared ? 0 : NP * kQ * VB;  // one buffer of c
  static constexpr int kW = PW * kQ * VB;
  static constexpr int kW2 = DG ? kW : 0;
  static constexpr int kS = PS * VB * KS;
  static constexpr int kT = PT * VB * KS;
  static constexpr int kLds = 160 * 1024;                         // of a CU
  static constexpr int kRows = kB + kC;                           // one buffer of rows
  static constexpr int kRest = kW + kW2 + kS + kT;                // one of weighted c and state
  static constexpr int bytes(int rows, int rest) { return 2 * (rows * kRows + rest * kRest) + (DG ? 1024 : 0); }
  // buffers of each, as the LDS allows.  Where one of the weighted c and the state
  // lets two blocks into a CU, that is worth more than a second buffer (bf16, 32
  // columns; 8 x 2048 x 24 heads of 128 x 128: 150 to 157 us against 169).
  static constexpr int kRestLds = NP == 1 && !DG && VB == 32 && 2 * bytes(2, 1) <= kLds ? kLds / 2 : kLds;
  static constexpr int NREST = !STATE && bytes(2, 2) <= kRestLds ? 2 : 1;
  static constexpr int NROWS = (STATE ? 2 : 1) * bytes(2, NREST) <= kLds ? 2 : 1;
  // b's rows are only read up to the scores; with two of c's, group B writes the
  // next chunk's while group A multiplies the scores with c
  static constexpr int NC = NROWS == 2 ? 2 : (!STATE && !kShared && bytes(1, 1) + 2 * kC <= kLds ? 2 : 1);
  static constexpr int kBytes = bytes(NROWS, NREST) + 2 * (NC - NROWS) * kC;
  static constexpr bool kFits = kBytes <= kLds;
  static_assert(!kShared || (NREST == 1 && NROWS == 1 && NP * kQ * VB <= VB * KS), "c in T's last part");
  // Waves of a group: eight for 64 columns, where a block has its CU to itself
  // and only more waves of its own hide its latencies.  WVA or WVB of them lie
  // along the columns v; group B's others along the rows kappa, group A's along
  // the four token blocks.
  static constexpr int NW = (VB >= 64 && !STATE && !DG) || VB == 128 ? 8 : 4;
  static constexpr int WVA = NW / 4;                // group A has a wave for every token block
  static constexpr int WVB = KP == 96 ? 2 : WVA;    // and 96 rows are three tiles for each of two waves
  static constexpr int NVA = VB / 16 / WVA;         // column tiles of a wave
  static constexpr int NVB = VB / 16 / WVB;
  static constexpr int JK = KP / 16 / (NW / WVB);   // row tiles of the state of a group B wave
  static constexpr int kGroup = 64 * NW;
  static constexpr int kThreads = STATE ? kGroup : 2 * kGroup;
  // waves per SIMD that the registers are shared out for: what the LDS lets in
  static constexpr int kWaves = STATE ? ((NW == 8 ? 2 : 4) * kBytes <= kLds ? 4 : (2 * kBytes <= kLds ? 2 : 1))
                                      : (NW == 8 || 2 * kBytes <= kLds ? 4 : 2);
};

__device__ __forceinline__ uint64_t low_bits(int n) {
  return n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// lam^e for e >= 0 (1 at e = 0 also where lam is 0)
__device__ __forceinline__ float power(float g2, int e) {
  return e == 0 ? 1.0f : exp2_hw(g2 * (float)e);
}

template <int NP, int KP, int VB, bool REV, bool DG, bool STATE>
__global__ __launch_bounds__((Shape<NP, KP, VB, DG, STATE>::kThreads), (Shape<NP, KP, VB, DG, STATE>::kWaves))
void walk_kernel(const WalkArgs p) {
  typedef typename Io<NP>::T T;
  typedef Shape<NP, KP, VB, DG, STATE> Sh;
  constexpr int ES = sizeof(T);
  constexpr int EPP = 16 / ES;                 // elements of a 16-byte piece
  constexpr int PRB = KP / EPP;                // pieces in a row of b
  constexpr int PRC = VB / EPP;                // pieces in a row of c
  constexpr int RB = kQ * PRB / Sh::kGroup;    // pieces of b per thread of group B
  constexpr int RC = kQ * PRC / Sh::kGroup;
  constexpr int PB = KP == 96 ? 8 : PRB;       // pieces of a row of b that threads lie along
  constexpr int RR = kQ * PB / Sh::kGroup;     // rows of b per thread
  constexpr int NK = KP / 32;                  // k-steps of a . b
  constexpr int KS = Sh::KS;
  constexpr int NROWS = Sh::NROWS, NC = Sh::NC, NREST = Sh::NREST;
  static_assert(RB >= 1 && RC >= 1 && Sh::NVA >= 1 && Sh::NVB >= 1 && Sh::JK >= 1, "tile too small");
  static_assert(NP == 3 || Sh::NVA % 2 == 0, "bf16 outputs leave two tiles at a time");

  __shared__ __align__(16) __bf16 lds[NROWS * Sh::kB + NC * Sh::kC + NREST * Sh::kRest];
  // chunk i's rows of b, of c and the rest (c weighted for S, for T; parts of S, of T)
  constexpr int kCw2 = Sh::kW, kSs = kCw2 + Sh::kW2, kTs = kSs + Sh::kS;
  auto b_at = [&](int i) { return lds + (NROWS == 2 ? (i & 1) * Sh::kB : 0); };
  auto c_at = [&](int i) {
    return lds + NROWS * Sh::kB + (Sh::kShared ? kTs + (Sh::PT - 1) * VB * KS : NC == 2 ? (i & 1) * Sh::kC : 0);
  };
  auto rest_at = [&](int i) {
    return lds + NROWS * Sh::kB + NC * Sh::kC + (NREST == 2 ? (i & 1) * Sh::kRest : 0);
  };

  // Consecutive block ids go round-robin to the 8 XCDs; each XCD gets a
  // contiguous run of (entry, head, span, slice), so the slices that read the
  // same a and b meet in its L2.
  const uint32_t per = (p.nblk + 7u) / 8u;
  const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x;  // y: more blocks than x holds
  const uint32_t logical = (id % 8u) * per + id / 8u;
  if (id / 8u >= per || logical >= p.nblk) return;
  uint32_t rest = logical;
  const int sl = (int)(rest % (uint32_t)p.nsl);
  rest /= (uint32_t)p.nsl;
  const int span = (int)(rest % (uint32_t)p.nspan_run);
  rest /= (uint32_t)p.nspan_run;
  const int h = (int)(rest % (uint32_t)p.H);
  const int b = (int)(rest / (uint32_t)p.H);

  constexpr int GT = Sh::kGroup;
  const int tid = threadIdx.x % GT, lane = tid & 63;  // within the group
  const bool group_a = !STATE && __builtin_amdgcn_readfirstlane((int)threadIdx.x / GT) == 0;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lk = lane >> 4;
  const int g4 = lane >> 4, kk = (lane & 15) >> 2, qq = lane & 3;  // of the transposing reads
  const int K = p.K, V = p.V;
  const int v0 = sl * VB;
  const float g2 = p.log_decay[h] * kLog2e;

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
  // the chunks of the span that hold real tokens, in the walk's order
  const int first = REV ? (i0 > nc - nlive ? i0 : nc - nlive) : i0;
  const int last = REV ? i1 : (i1 < nlive ? i1 : nlive);

  // One sequence and head of a tensor of (L, heads, width): byte offsets
  // within a chunk fit 32 bits (the launch bounds heads * width).
  const int64_t bL = (int64_t)b * L;
  const int64_t bh = (int64_t)b * p.H + h;
  const int64_t state_elems = (int64_t)K * V;
  const uint32_t rsc = (uint32_t)p.Hc * V * ES;
  auto rows_of = [&](const char* base, int64_t t0, uint32_t stride, int n, int width) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)(base + t0 * stride), (short)0,
                                             n ? (int)((uint32_t)(n - 1) * stride + (uint32_t)width * ES) : 0,
                                             kBufferFlags);
  };
  auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint32_t o) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)o, 0, 0));
  };
  // the document starts of a chunk, one byte per token (without a branch: an
  // empty range reads zeros)
  auto load_starts = [&](int c) -> uint32_t {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.reset + bL + (int64_t)c * kQ), (short)0, p.reset ? live_in(c) : 0, kBufferFlags);
    return __builtin_amdgcn_raw_buffer_load_b8(r, lane, 0, 0);
  };

  float dg = 0.0f;       // of one chunk
  double dg_sum = 0.0;   // its sums cancel over the chunks, so they are held in 64 bits

  if (!STATE && group_a) {
    // ================================================== group A: the outputs
    constexpr int NVW = Sh::NVA;
    constexpr int PP = NP == 3 ? 3 : 2;  // parts of the scores that lead to out
    constexpr int RA = NP == 1 ? NK : 2 * NK;
    const int vw = 16 * NVW * (w % Sh::WVA);                             // first column of the wave in the slice
    const int blk = __builtin_amdgcn_readfirstlane(w / Sh::WVA);         // its token block
    const int t = 16 * blk + lr;                                        // this lane's token in a chunk
    const uint32_t rsa = (uint32_t)p.Ha * K * ES;
    const char* const pa = (const char*)p.a + (bL * p.Ha + h / (p.H / p.Ha)) * (int64_t)K * ES;
    const char* const px = DG ? (const char*)p.x + ((bL * p.Hc + h / (p.H / p.Hc)) * (int64_t)V + v0) * ES : nullptr;

    u32x4 rA[RA];
    uint32_t rR = 0;
    // Two loads cover 128 bytes of the block's 16 rows, 8 whole row pieces each:
    // load u, lane (lk, lr) takes row 8 u + lr % 8, 16 bytes at 16 (2 lk +
    // lr / 8).  take_a trades halves between the two.
    constexpr int kPairElems = 128 / ES;
    auto load_a = [&](int c) {
      const __amdgpu_buffer_rsrc_t r = rows_of(pa, (int64_t)c * kQ, rsa, live_in(c), K);
      const int piece = 2 * lk + (lr >> 3);
#pragma unroll
      for (int j = 0; j < RA; ++j) {
        const uint32_t row = (uint32_t)(16 * blk + 8 * (j % 2) + (lr & 7));
        const int col = kPairElems * (j / 2) + EPP * piece;
        rA[j] = load16(r, col < K ? row * rsa + (uint32_t)(col * ES) : kOutside);
      }
      rR = load_starts(c);
    };
    bf16x8 aF[NK][NP];
    uint64_t starts = 0;
    int edge = 0;  // where token t's document begins; backwards, where the next one does
    auto take_a = [&]() {
      starts = __ballot((rR & 0xffu) != 0);
      if (starts) {
        const uint64_t m = REV ? (starts >> t) >> 1 : starts & low_bits(t + 1);
        edge = REV ? (m ? t + 1 + __builtin_ctzll(m) : kQ) : (m ? 63 - __builtin_clzll(m) : -1);
      }
#pragma unroll
      for (int j = 0; j < RA / 2; ++j) {
        // pieces 2 lk and 2 lk + 1 of row lr: within each 16 lanes, the upper
        // half of one comes from the other load 8 lanes down, the lower half
        // of the other 8 lanes up
        u32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r0 = (int)rA[2 * j][i], r1 = (int)rA[2 * j + 1][i];
          lo[i] = (uint32_t)__builtin_amdgcn_update_dpp(r0, r1, 0x118, 0xf, 0xc, false);  // row_shr:8
          hi[i] = (uint32_t)__builtin_amdgcn_update_dpp(r1, r0, 0x108, 0xf, 0x3, false);  // row_shl:8
        }
        if constexpr (NP == 1) {
          aF[2 * j][0] = __builtin_bit_cast(bf16x8, lo);
          aF[2 * j + 1][0] = __builtin_bit_cast(bf16x8, hi);
        } else {
          uint32_t pt[4][3];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            split2<3>(__uint_as_float(lo[2 * i]), __uint_as_float(lo[2 * i + 1]), pt[i]);
            split2<3>(__uint_as_float(hi[2 * i]), __uint_as_float(hi[2 * i + 1]), pt[2 + i]);
          }
#pragma unroll
          for (int e = 0; e < 3; ++e)
            aF[j][e] = __builtin_bit_cast(bf16x8, u32x4{pt[0][e], pt[1][e], pt[2][e], pt[3][e]});
        }
      }
    };

    // lane constants of the intra-chunk weights, of token t = 16 W + lr and
    // s = 16 sb + 4 lk + i: on the diagonal block lam^|lr - 4 lk - i|, m blocks
    // away lam^(16 m - 16) times the weight one block away
    float wd[4], w1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = REV ? 4 * lk + i - lr : lr - 4 * lk - i;  // tokens from s to t along the walk
      wd[i] = e >= 0 ? p.s_intra * power(g2, e) : 0.0f;
      w1[i] = p.s_intra * power(g2, 16 + e);  // e > -16
    }
    const float lam16 = power(g2, 16), lam32 = power(g2, 32);
    // the weight of the state at this lane's token of a full chunk
    const float wi_full = p.s_inter * power(g2, REV ? kQ - 1 - t : t + 1);

    f32x4 acc[NVW], acc2[DG ? NVW : 1];
    u32x4 rX[DG ? NVW : 1];

    // acc = W a_t (rows v, columns t), weighted
    auto state_part = [&](int n, const __bf16* Ss, const __bf16* Ts) {
#pragma unroll
      for (int vt = 0; vt < NVW; ++vt) {
        acc[vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (DG) acc2[vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        bf16x8 sF[NVW][Sh::PS > 0 ? Sh::PS : 1], tF[DG ? NVW : 1][Sh::PT > 0 ? Sh::PT : 1];
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          const int at = (vw + 16 * vt + lr) * KS + sw<KP>(lr, kcol<NP>(k, lk));
#pragma unroll
          for (int e = 0; e < Sh::PS; ++e) sF[vt][e] = *(const bf16x8*)(Ss + e * VB * KS + at);
          if constexpr (DG) {
#pragma unroll
            for (int e = 0; e < Sh::PT; ++e) tF[vt][e] = *(const bf16x8*)(Ts + e * VB * KS + at);
          }
        }
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          acc[vt] = mfma_parts(sF[vt], aF[k], acc[vt]);
          if constexpr (DG) acc2[vt] = mfma_parts(tF[vt], aF[k], acc2[vt]);
        }
      }
      settle(acc);
      if constexpr (DG) settle(acc2);
      const int je = REV ? n - 1 - t : t + 1;
      const float wi = REV && n < kQ ? p.s_inter * power(g2, je > 0 ? je : 0) : wi_full;
#pragma unroll
      for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (DG) acc2[vt][i] = wi * (acc2[vt][i] + (float)je * acc[vt][i]);
          acc[vt][i] *= wi;
        }
      if (n < kQ || starts) {
        const bool from = t < n && (!starts || edge == (REV ? kQ : -1));
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (DG) acc2[vt][i] = from ? acc2[vt][i] : 0.0f;
            acc[vt][i] = from ? acc[vt][i] : 0.0f;
          }
      }
    };

    // The chunk's own part for token block W (uniform in a wave): scores
    // transposed (s by t), weighted, and as they stand, two 16-token blocks of
    // s at a time, the operand of the product with c.
    auto chunk_part = [&](auto Wc, const __bf16* Bs, const __bf16* Cs) {
      constexpr int W = decltype(Wc)::value;
      f32x4 g[4];
#pragma unroll
      for (int sb = 0; sb < 4; ++sb) g[sb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int sb = REV ? W : 0; sb <= (REV ? 3 : W); ++sb) {
          bf16x8 bF[NP];
#pragma unroll
          for (int e = 0; e < NP; ++e)
            bF[e] = *(const bf16x8*)(Bs + e * kQ * KS + (16 * sb + lr) * KS + sw<KP>(lr, kcol<NP>(k, lk)));
          g[sb] = mfma_parts(bF, aF[k], g[sb]);
        }
      settle(g);
      if (starts) {  // group B clears rows of b (clear_cut)
        lds_barrier();
        lds_barrier();
      }
      // Group B may write the rest.  Here the two halves of a chunk are alike in
      // both groups: staging and update beside state part and scores (f32, 128
      // keys: 63 us for 3 x 1537 x 12 heads; with the barrier before the scores 78).
      if ((NREST == 1 && NC == 2) || Sh::kShared) lds_barrier();
#pragma unroll
      for (int pair = REV ? W / 2 : 0; pair <= (REV ? 1 : W / 2); ++pair) {
        const int ra = 32 * pair + 4 * g4 + kk, rb = ra + 16;
        bf16x8 cF[NVW][NP];
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
          for (int e = 0; e < NP; ++e)
            cF[vt][e] = join(tr_read(Cs + e * kQ * VB + ra * VB + swc<VB>(ra, vw + 16 * vt + 4 * qq)),
                             tr_read(Cs + e * kQ * VB + rb * VB + swc<VB>(rb, vw + 16 * vt + 4 * qq)));
        uint32_t pw[2][2][PP], pw2[2][2][DG ? 3 : 1];  // [block][half][part]
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int sb = 2 * pair + u;
          const int m = REV ? sb - W : W - sb;  // blocks from s to t
          if (m < 0) {
#pragma unroll
            for (int e = 0; e < PP; ++e) pw[u][0][e] = pw[u][1][e] = 0;
            if constexpr (DG) {
#pragma unroll
              for (int e = 0; e < 3; ++e) pw2[u][0][e] = pw2[u][1][e] = 0;
            }
            continue;
          }
          float x[4], x2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float y = g[sb][i] * (m == 0 ? wd[i] : w1[i]);
            if (m == 2) y *= lam16;
            if (m == 3) y *= lam32;
            // a token that t does not see leaves nothing, whatever its score (a NaN in
            // its row of c does: the product takes the whole chunk)
            if (m == 0) y = (REV ? 4 * lk + i >= lr : 4 * lk + i <= lr) ? y : 0.0f;
            x[i] = y;
          }
          if (starts) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int s = 16 * sb + 4 * lk + i;
              x[i] = (REV ? s < edge : s >= edge) ? x[i] : 0.0f;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x2[i] = DG ? x[i] * (float)(16 * m + (REV ? 4 * lk + i - lr : lr - 4 * lk - i)) : 0.0f;
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
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          acc[vt] = mfma_parts(cF[vt], pF, acc[vt]);
          if constexpr (DG) acc2[vt] = mfma_parts(cF[vt], pF2, acc2[vt]);
        }
      }
      settle(acc);
      if constexpr (DG) settle(acc2);
    };

    if (first < last) {
      load_a(chunk_of(first));
      take_a();
      if (first + 1 < last) load_a(chunk_of(first + 1));
    }
    lds_barrier();
    for (int i = first; i < last; ++i) {
      const int c = chunk_of(i), n = live_in(c);
      const __bf16 *const Bs = b_at(i), *const Cs = c_at(i);
      const __bf16* const rest = rest_at(i);
      if constexpr (DG) {  // x of this lane's outputs
        const __amdgpu_buffer_rsrc_t r = rows_of(px, (int64_t)c * kQ, rsc, n, V - v0);
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          const int col = vw + 16 * vt + 4 * lk;
          const uint32_t o = v0 + col < V ? (uint32_t)t * rsc + (uint32_t)col * ES : kOutside;
          if constexpr (NP == 1) {
            const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)o, 0, 0));
            rX[vt] = u32x4{x[0], x[1], 0u, 0u};
          } else {
            rX[vt] = load16(r, o);
          }
        }
      }
      state_part(n, rest + kSs, rest + kTs);
      if (Sh::kShared) lds_barrier();  // group B may write c over T's last part
      if (blk == 0) chunk_part(std::integral_constant<int, 0>{}, Bs, Cs);
      else if (blk == 1) chunk_part(std::integral_constant<int, 1>{}, Bs, Cs);
      else if (blk == 2) chunk_part(std::integral_constant<int, 2>{}, Bs, Cs);
      else chunk_part(std::integral_constant<int, 3>{}, Bs, Cs);
      if constexpr (DG) {
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = NP == 1 ? ((e & 1) ? hi_bf(rX[vt][e / 2]) : lo_bf(rX[vt][e / 2]))
                                    : __uint_as_float(rX[vt][e]);
            dg = t < n ? fmaf(acc2[vt][e], x, dg) : dg;
          }
        dg_sum += (double)dg;
        dg = 0.0f;
      }
      if (NC == 1) lds_barrier();  // group B may write everything
      // the next chunk's a, from loads a chunk old, and the loads after it
      // (before the stores, so that no wait for loads is one for stores)
      if (i + 1 < last) {
        take_a();
        if (i + 2 < last) load_a(chunk_of(i + 2));
      }
      // out rows of real tokens, and zeros at padding inside the chunk
      {
        const bool wide = NP == 3 || p.out_f32;
        const uint32_t oes = wide ? 4u : 2u;
        const uint32_t rso = (uint32_t)p.H * V * oes;
        const int64_t left = L - (int64_t)c * kQ < kQ ? L - (int64_t)c * kQ : kQ;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void*)((char*)p.out + (((bL + (int64_t)c * kQ) * p.H + h) * V + v0) * (int64_t)oes), (short)0,
            (int)((uint32_t)(left - 1) * rso + (uint32_t)(V - v0) * oes), kBufferFlags);
        if (t >= n) {
#pragma unroll
          for (int vt = 0; vt < NVW; ++vt) acc[vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        if (wide) {
#pragma unroll
          for (int vt = 0; vt < NVW; ++vt) {
            const int v = vw + 16 * vt + 4 * lk;
            const int at = v0 + v < V ? (int)((uint32_t)t * rso + (uint32_t)v * 4u) : (int)kOutside;
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[vt]), r, at, 0, kNt);
          }
        } else if constexpr (NP == 1) {
          // lanes hold 4 columns of each of two tiles; the swaps (odd rows of
          // 16 lanes of one operand with the even rows of the other) leave 8
          // columns of one, so that a store writes 64 bytes of each row
#pragma unroll
          for (int vt = 0; vt < NVW; vt += 2) {
            const int v = vw + 16 * (vt + (lk & 1)) + 8 * (lk >> 1);
            const int at = v0 + v < V ? (int)((uint32_t)t * rso + (uint32_t)v * 2u) : (int)kOutside;
            const f32x4 o0 = acc[vt], o1 = acc[vt + 1];
            const auto s0 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(o0[0], o0[1]), pack_bf16x2(o1[0], o1[1]), false, false);
            const auto s1 = __builtin_amdgcn_permlane16_swap(pack_bf16x2(o0[2], o0[3]), pack_bf16x2(o1[2], o1[3]), false, false);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{s0[0], s1[0], s0[1], s1[1]}, r, at, 0, kNt);
          }
        }
      }
      lds_barrier();
    }
    // padding rows of the span that no chunk above held: zeros
    const int ca = chunk_of(REV ? i1 - 1 : i0), cb = chunk_of(REV ? i0 : i1 - 1) + 1;
    const int64_t z0 = ((int64_t)(ca > nlive ? ca : nlive)) * kQ;
    const int64_t z1 = (int64_t)cb * kQ < L ? (int64_t)cb * kQ : L;
    const int cols = V - v0 < VB ? V - v0 : VB;
    for (int64_t q = tid; q < (z1 - z0) * (VB / 4); q += GT) {
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
  } else {
    // ======================================= group B: b, c and the state
    constexpr int NVW = Sh::NVB;
    const uint32_t rsb = (uint32_t)p.Hb * K * ES;
    const char* const pb = (const char*)p.b + (bL * p.Hb + h / (p.H / p.Hb)) * (int64_t)K * ES;
    const char* const pc = (const char*)p.c + ((bL * p.Hc + h / (p.H / p.Hc)) * (int64_t)V + v0) * ES;
    // lam^64 in two parts: its error, also that of rounding it to fp32, would
    // come in once per chunk, and 100 chunks of a slow decay made 1e-6 of it
    const double lam64d = exp(64.0 * (double)p.log_decay[h]);
    const float lam64 = (float)lam64d, lam64_lo = lam64 > 0.0f ? (float)(lam64d - (double)lam64) : 0.0f;

    u32x4 rB[RB], rC[RC];
    uint32_t rR = 0;
    const int rowB = tid / PB, pieceB = tid % PB;
    // piece j of this thread
    auto b_row = [&](int j) { return rowB + (RR == RB ? j : j % RR) * (GT / PB); };
    auto b_piece = [&](int j) { return RR == RB ? pieceB : pieceB + j / RR * PB; };
    const int rowC = tid / PRC, pieceC = tid % PRC;
    auto load_bc = [&](int c) {
      const int n = live_in(c);
      const __amdgpu_buffer_rsrc_t qb = rows_of(pb, (int64_t)c * kQ, rsb, n, K);
      const __amdgpu_buffer_rsrc_t qc = rows_of(pc, (int64_t)c * kQ, rsc, n, V - v0);
      const bool inb = pieceB * EPP < K, inc = v0 + pieceC * EPP < V;
#pragma unroll
      for (int j = 0; j < RB; ++j)
        rB[j] = load16(qb, (RR == RB ? inb : b_piece(j) * EPP < K) ? (uint32_t)b_row(j) * rsb + b_piece(j) * 16u : kOutside);
#pragma unroll
      for (int j = 0; j < RC; ++j)
        rC[j] = load16(qc, inc ? (uint32_t)(rowC + j * (GT / PRC)) * rsc + pieceC * 16u : kOutside);
      rR = load_starts(c);
    };

    uint64_t starts = 0;  // of the staged chunk
    // the weight of this thread's rows of a full chunk in the state at its end
    float w_full[RC];
#pragma unroll
    for (int j = 0; j < RC; ++j) {
      const int row = rowC + j * (GT / PRC);
      w_full[j] = p.s_state * power(g2, REV ? row + 1 : kQ - 1 - row);
    }
    u32x4 cC[RC];          // c of the chunk being staged
    uint32_t cR = 0;
    auto c_value = [&](int j, int i) {
      return NP == 1 ? ((i & 1) ? hi_bf(cC[j][i / 2]) : lo_bf(cC[j][i / 2])) : __uint_as_float(cC[j][i % 4]);
    };
    // whether row's document reaches the chunk's end (in the walk's direction)
    auto to_end = [](uint64_t s, int row) { return REV ? (s & low_bits(row + 1)) == 0 : ((s >> row) >> 1) == 0; };
    // the weighted c of the loaded chunk
    auto stage_weighted = [&](int n, __bf16* Cw, __bf16* Cw2) {
      starts = __ballot((cR & 0xffu) != 0);
#pragma unroll
      for (int j = 0; j < RC; ++j) {
        const int row = rowC + j * (GT / PRC), col = pieceC * EPP;
        const int at = row * VB + swc<VB>(row, col);
        const int e = REV ? row + 1 : n - 1 - row;
        float wt = w_full[j];
        bool in = true;
        if (n < kQ) {
          in = row < n;
          if (!REV) wt = in ? p.s_state * power(g2, e) : 0.0f;
        }
        if (starts) in = in && to_end(starts, row);
        wt = in ? wt : 0.0f;
#pragma unroll
        for (int which = 0; which < (DG ? 2 : 1); ++which) {
          const float wq = which == 0 ? wt : wt * (float)(in ? e : 0);
          __bf16* const d = (which == 0 ? Cw : Cw2) + at;
          uint32_t pt[EPP / 2][3];
#pragma unroll
          for (int i = 0; i < EPP / 2; ++i) split2<3>(c_value(j, 2 * i) * wq, c_value(j, 2 * i + 1) * wq, pt[i]);
          if (starts) {  // as b's rows in clear_cut
#pragma unroll
            for (int i = 0; i < EPP / 2; ++i)
#pragma unroll
              for (int q = 0; q < 3; ++q) pt[i][q] = in ? pt[i][q] : 0u;
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
    };
    // rows of the loaded chunk: b's and c's, or c's alone, late (kShared)
    constexpr std::true_type kLate{};
    constexpr std::false_type kOnTime{};
    auto stage_rows = [&](__bf16* Bs, __bf16* Cs, auto late) {
      if constexpr (!late) {
#pragma unroll
        for (int j = 0; j < RC; ++j) cC[j] = rC[j];
        cR = rR;
        if constexpr (STATE) {  // b is only read for the state (see clear_cut)
          const uint64_t s = __ballot((rR & 0xffu) != 0);
          if (s) {
#pragma unroll
            for (int j = 0; j < RB; ++j)
              if (!to_end(s, b_row(j))) rB[j] = u32x4{0u, 0u, 0u, 0u};
          }
        }
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          const int row = b_row(j), col = b_piece(j) * EPP;
          __bf16* const d = Bs + row * KS + sw<KP>(row, col);
          if constexpr (NP == 1) {
            *(u32x4*)d = rB[j];
          } else {
            uint32_t p0[3], p1[3];
            split2<3>(__uint_as_float(rB[j][0]), __uint_as_float(rB[j][1]), p0);
            split2<3>(__uint_as_float(rB[j][2]), __uint_as_float(rB[j][3]), p1);
#pragma unroll
            for (int q = 0; q < 3; ++q) *(u32x2*)(d + q * kQ * KS) = u32x2{p0[q], p1[q]};
          }
        }
      }
      if constexpr (!STATE && late == Sh::kShared) {
#pragma unroll
        for (int j = 0; j < RC; ++j) {
          const int row = rowC + j * (GT / PRC), col = pieceC * EPP;
          __bf16* const d = Cs + row * VB + swc<VB>(row, col);
          if constexpr (NP == 1) {
            *(u32x4*)d = cC[j];
          } else {
            uint32_t p0[3], p1[3];
            split2<3>(c_value(j, 0), c_value(j, 1), p0);
            split2<3>(c_value(j, 2), c_value(j, 3), p1);
#pragma unroll
            for (int q = 0; q < 3; ++q) *(u32x2*)(d + q * kQ * VB) = u32x2{p0[q], p1[q]};
          }
        }
      }
    };

    // A token that does not reach the chunk's end leaves nothing in the state,
    // whatever it holds.  A weight of zero is not enough for a NaN, so in a chunk
    // with document starts b's rows are cleared too, once the scores are done (3 x
    // 1537 tokens of 12 heads in documents of 500, fp32: 314 -> 327 us; clearing the
    // operands in registers 321, but 2 to 8% of every walk without documents).
    auto clear_cut = [&](__bf16* Bs) {
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int row = b_row(j), col = b_piece(j) * EPP;
        __bf16* const d = Bs + row * KS + sw<KP>(row, col);
        if (!to_end(starts, row)) {
          if constexpr (NP == 1) {
            *(u32x4*)d = u32x4{0u, 0u, 0u, 0u};
          } else {
#pragma unroll
            for (int q = 0; q < 3; ++q) *(u32x2*)(d + q * kQ * KS) = u32x2{0u, 0u};
          }
        }
      }
    };

    // the state, fp32, in the matrix cores' result layout: lane value i of tile
    // (j, vt) is W[v = vw + 16 vt + lr][kappa = kw + 16 j + 4 lk + i]
    constexpr int JK = Sh::JK;
    const int vw = 16 * NVW * (w % Sh::WVB), kw = 16 * JK * (w / Sh::WVB);
    f32x4 S[JK][NVW], D[DG ? JK : 1][DG ? NVW : 1];
#pragma unroll
    for (int j = 0; j < JK; ++j)
#pragma unroll
      for (int vt = 0; vt < NVW; ++vt) {
        S[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (DG) D[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    auto for_state = [&](auto&& f) {
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          const int v = v0 + vw + 16 * vt + lr, k = kw + 16 * j + 4 * lk;
          if (v < V && k < K) f(j, vt, v, k);
        }
    };
    auto put_state = [&](__bf16* Ss, __bf16* Ts) {
      if constexpr (!STATE) {
#pragma unroll
        for (int j = 0; j < JK; ++j)
#pragma unroll
          for (int vt = 0; vt < NVW; ++vt) {
            const int at = (vw + 16 * vt + lr) * KS + sw<KP>(lr, kw + 16 * j + 4 * lk);
            {
              uint32_t p0[Sh::PS], p1[Sh::PS];
              split2<Sh::PS>(S[j][vt][0], S[j][vt][1], p0);
              split2<Sh::PS>(S[j][vt][2], S[j][vt][3], p1);
#pragma unroll
              for (int q = 0; q < Sh::PS; ++q) *(u32x2*)(Ss + q * VB * KS + at) = u32x2{p0[q], p1[q]};
            }
            if constexpr (DG) {
              uint32_t p0[Sh::PT], p1[Sh::PT];
              split2<Sh::PT>(D[j][vt][0], D[j][vt][1], p0);
              split2<Sh::PT>(D[j][vt][2], D[j][vt][3], p1);
#pragma unroll
              for (int q = 0; q < Sh::PT; ++q) *(u32x2*)(Ts + q * VB * KS + at) = u32x2{p0[q], p1[q]};
            }
          }
      }
    };
    // The state at the walk's end of the staged chunk.  Where its last bits matter
    // (fp32 results, and the state and T behind the log-decay's gradient), the
    // chunk's own part is added up by itself: a slow head's state is large beside
    // it, and each product that adds to it rounds to its size, 6 or 12 times a chunk
    // (T after 2000 tokens with a memory of 4096: 3.8e-7 to 6.4e-7 instead of 1.2e-7
    // to 1.9e-7).  Rows of 256 then leave the two steps of the products a loop: unrolled,
    // the kernel outgrows the instruction cache (2 x 2048 x 24 heads of 64 x 256, bf16,
    // with all gradients 381 us against 341).
    constexpr bool APART = DG || NP == 3;
    constexpr bool ROLL = APART && KP == 256;
    auto update = [&](int n, const __bf16* Bs, const __bf16* Cw, const __bf16* Cw2) {
      const bool cut = starts != 0;
      const float d = n == kQ ? lam64 : power(g2, n), dl = n == kQ ? lam64_lo : 0.0f;
      const float nf = (float)n;
      if constexpr (!APART) {
#pragma unroll
        for (int j = 0; j < JK; ++j)
#pragma unroll
          for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][vt][i] = fmaf(S[j][vt][i], d, S[j][vt][i] * dl);
        if (cut) {
#pragma unroll
          for (int j = 0; j < JK; ++j)
#pragma unroll
            for (int vt = 0; vt < NVW; ++vt) S[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
      }
      f32x4 P[JK][NVW], PD[DG ? JK : 1][DG ? NVW : 1];
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          P[j][vt] = APART ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : S[j][vt];
          if constexpr (DG) PD[j][vt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
      auto settle_all = [&]() {
#pragma unroll
        for (int j = 0; j < JK; ++j) {
          settle(P[j]);
          if constexpr (DG) settle(PD[j]);
        }
      };
#pragma unroll(ROLL ? 1 : 2)
      for (int ks = 0; ks < 2; ++ks) {
        const int ra = 32 * ks + 8 * g4 + kk, rb = ra + 4;
        bf16x8 bF[JK][NP];
#pragma unroll
        for (int j = 0; j < JK; ++j)
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            const int col = kw + 16 * j + 4 * qq;
            bF[j][e] = join(tr_read(Bs + e * kQ * KS + ra * KS + sw<KP>(ra, col)),
                            tr_read(Bs + e * kQ * KS + rb * KS + sw<KP>(rb, col)));
          }
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt) {
          const int col = vw + 16 * vt + 4 * qq;
          bf16x8 cF[3], cF2[DG ? 3 : 1];
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            const int at = e * kQ * VB;
            cF[e] = join(tr_read(Cw + at + ra * VB + swc<VB>(ra, col)),
                         tr_read(Cw + at + rb * VB + swc<VB>(rb, col)));
            if constexpr (DG)
              cF2[e] = join(tr_read(Cw2 + at + ra * VB + swc<VB>(ra, col)),
                            tr_read(Cw2 + at + rb * VB + swc<VB>(rb, col)));
          }
#pragma unroll
          for (int j = 0; j < JK; ++j) {
            P[j][vt] = mfma_parts(bF[j], cF, P[j][vt]);
            if constexpr (DG) PD[j][vt] = mfma_parts(bF[j], cF2, PD[j][vt]);
          }
        }
        if constexpr (ROLL) settle_all();  // before the loop's branch
      }
      settle_all();
#pragma unroll
      for (int j = 0; j < JK; ++j)
#pragma unroll
        for (int vt = 0; vt < NVW; ++vt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (DG) {
              const float t = D[j][vt][i] + nf * S[j][vt][i];
              D[j][vt][i] = cut ? PD[j][vt][i] : fmaf(t, d, fmaf(t, dl, PD[j][vt][i]));
            }
            const float s = S[j][vt][i];
            S[j][vt][i] = !APART || cut ? P[j][vt][i] : fmaf(s, d, fmaf(s, dl, P[j][vt][i]));
          }
    };

    if (first < last) load_bc(chunk_of(first));
    if constexpr (!STATE) {
      if (p.init) {
        const float* s0 = p.init + bh * state_elems;
        for_state([&](int j, int vt, int v, int k) {
#pragma unroll
          for (int i = 0; i < 4; ++i) S[j][vt][i] = s0[v * p.state_sv + (k + i) * p.state_sk];
        });
      }
      // the states that the pieces of the walk before this span add, in order; U
      // of them loaded at once (one at a time, each costs a trip to memory: 412 us
      // against 351 for 2 x 14447 tokens of 2 heads, 128 x 80, with all gradients)
      constexpr int U = JK * NVW * (DG ? 2 : 1) <= 4 ? 4 : 2;
      const int np = i0 / p.piece_chunks;
      // the decay over a whole piece in two parts, as over a chunk (one fp32 factor
      // for each of hundreds of pieces: 1.5e-5 of a slow decay)
      const int64_t whole = (int64_t)p.piece_chunks * kQ;
      const double lampd = np > 0 ? exp((double)whole * (double)p.log_decay[h]) : 0.0;
      const float lamp = (float)lampd, lamp_lo = lamp > 0.0f ? (float)(lampd - (double)lamp) : 0.0f;
      for (int m = 0; m < np; m += U) {
        f32x4 av[U][JK][NVW], tv[U][DG ? JK : 1][DG ? NVW : 1];
        int cut[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int mu = m + u < np ? m + u : np - 1;
          const float* loc = p.ws + ((int64_t)mu * p.batch * p.H + bh) * (DG ? 2 : 1) * state_elems;
          cut[u] = p.piece_cut[(int64_t)mu * p.batch + b];
#pragma unroll
          for (int j = 0; j < JK; ++j)
#pragma unroll
            for (int vt = 0; vt < NVW; ++vt) {
              const int v = v0 + vw + 16 * vt + lr, k = kw + 16 * j + 4 * lk;
              const int64_t at = v < V && k < K ? (int64_t)v * K + k : 0;  // the rest is not used
              av[u][j][vt] = *(const f32x4*)(loc + at);
              if constexpr (DG) tv[u][j][vt] = *(const f32x4*)(loc + state_elems + at);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (m + u >= np) break;
          // real tokens of the piece
          const int m0 = (m + u) * p.piece_chunks, m1 = m0 + p.piece_chunks - 1;
          const int64_t ca = chunk_of(REV ? m1 : m0), cb = chunk_of(REV ? m0 : m1) + 1;
          const int64_t hi = cb * kQ < len ? cb * kQ : len;
          const int64_t n = hi > ca * kQ ? hi - ca * kQ : 0;
          const float d = n == whole ? lamp : n == 0 ? 1.0f : exp2_hw(g2 * (float)n);
          const float dl = n == whole ? lamp_lo : 0.0f;
          for_state([&](int j, int vt, int, int) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (DG) {
                const float t = D[j][vt][i] + (float)n * S[j][vt][i];
                D[j][vt][i] = cut[u] ? tv[u][j][vt][i] : fmaf(t, d, fmaf(t, dl, tv[u][j][vt][i]));
              }
              S[j][vt][i] = cut[u] ? av[u][j][vt][i] : fmaf(S[j][vt][i], d, fmaf(S[j][vt][i], dl, av[u][j][vt][i]));
            }
          });
        }
      }
    }
    int any_start = 0;
    if (first < last) {
      stage_rows(b_at(first), c_at(first), kOnTime);
      if (first + 1 < last) load_bc(chunk_of(first + 1));
      __bf16* const rest = rest_at(first);
      stage_weighted(live_in(chunk_of(first)), rest, rest + kCw2);
      put_state(rest + kSs, rest + kTs);
    }
    lds_barrier();
    for (int i = first; i < last; ++i) {
      const __bf16* const rest = rest_at(i);
      __bf16* const next = rest_at(i + 1);
      const bool more = i + 1 < last;
      auto stage_next = [&]() {
        stage_rows(b_at(i + 1), c_at(i + 1), kOnTime);
        if (i + 2 < last) load_bc(chunk_of(i + 2));  // a chunk ahead of its use
      };
      any_start |= starts != 0;
      if (NROWS == 2 && more) stage_next();
      if constexpr (Sh::kShared) {
        lds_barrier();
        stage_rows(nullptr, c_at(i), kLate);
      }
      if constexpr (!STATE) {
        if (starts) {
          lds_barrier();
          clear_cut(b_at(i));
          lds_barrier();
        }
      }
      if constexpr (Sh::kShared) lds_barrier();
      update(live_in(chunk_of(i)), b_at(i), rest, rest + kCw2);
      if (NREST == 1) lds_barrier();  // what update read may be written
      if (NROWS == 1 && more) stage_next();
      if (more) {
        put_state(next + kSs, next + kTs);
        stage_weighted(live_in(chunk_of(i + 1)), next, next + kCw2);
      }
      lds_barrier();
    }

    if constexpr (STATE) {
      float* loc = p.ws + ((int64_t)span * p.batch * p.H + bh) * (DG ? 2 : 1) * state_elems;
      for_state([&](int j, int vt, int v, int k) {
        *(f32x4*)(loc + (int64_t)v * K + k) = S[j][vt];
        if constexpr (DG) *(f32x4*)(loc + state_elems + (int64_t)v * K + k) = D[j][vt];
      });
      if (h == 0 && sl == 0 && tid == 0) p.piece_cut[(int64_t)span * p.batch + b] = any_start;
    } else {
      const bool ends = span == p.nspan - 1;  // this block ends the walk
      if (ends && p.final_state) {
        float* fs = p.final_state + bh * state_elems;
        for_state([&](int j, int vt, int v, int k) { *(f32x4*)(fs + (int64_t)v * K + k) = S[j][vt]; });
      }
      if constexpr (DG) {
        if (ends && p.dlast) {  // <dlast, T after the last token>; dlast is K-major here
          const float* dl = p.dlast + bh * state_elems;
          for_state([&](int j, int vt, int v, int k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dg = fmaf(dl[(int64_t)(k + i) * V + v], D[j][vt][i], dg);
          });
        }
      }
    }
  }

  if constexpr (DG && !STATE) {
    // the block's sum, in a fixed order
    __shared__ double sums[2 * Sh::NW];
    dg_sum += (double)dg;  // <dlast, T>
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) dg_sum += __shfl_xor(dg_sum, m);
    if (lane == 0) sums[threadIdx.x >> 6] = dg_sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < 2 * Sh::NW; ++i) s += sums[i];
      p.dg_part[(int64_t)h * p.batch * p.nsl * p.nspan + ((int64_t)b * p.nsl + sl) * p.nspan + span] = s;
    }
  }
}

template <int NP, int KP, int VB>
hipError_t launch_walk(const WalkArgs& args, bool rev, bool dg, bool state, hipStream_t stream) {
  WalkArgs a = args;
  a.nspan_run = state ? a.pieces : a.nspan;
  if (state) a.span_chunks = a.piece_chunks;
  a.nsl = (a.V + VB - 1) / VB;
  const int64_t n = (int64_t)a.batch * a.H * a.nsl * a.nspan_run;
  if (n == 0) return hipSuccess;
  a.nblk = (uint32_t)n;
  // the kernels that a plan can choose: the outputs' walk takes 64 columns at
  // most, and 32 with the log-decay's gradient, whose state walk takes 64
#define SSM_WALK(REV, DG, STATE)                                                                      \
  do {                                                                                                \
    if constexpr (VB <= (STATE ? (DG ? 64 : 128) : (DG ? 32 : 64))) {                                 \
      static_assert(Shape<NP, KP, VB, DG, STATE>::kFits, "more than the LDS of a CU");                \
      constexpr int kThreads = Shape<NP, KP, VB, DG, STATE>::kThreads;                                \
      const Grid g = grid_of((n + 7) / 8 * 8, kThreads);                                              \
      walk_kernel<NP, KP, VB, REV, DG, STATE><<<dim3(g.x, g.more), dim3(kThreads), 0, stream>>>(a);   \
    } else {                                                                                          \
      return hipErrorInvalidValue;                                                                    \
    }                                                                                                 \
  } while (0)
  if (state && rev) SSM_WALK(true, false, true);
  else if (state && dg) SSM_WALK(false, true, true);
  else if (state) SSM_WALK(false, false, true);
  else if (rev) SSM_WALK(true, false, false);
  else if (dg) SSM_WALK(false, true, false);
  else SSM_WALK(false, false, false);
#undef SSM_WALK
  return hipGetLastError();
}

}  // namespace linattn
}  // namespace ssm66
