// linattn_launch.h -- internal interface of the linear-attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace ssm66 {
namespace linattn {

constexpr int kChunk = 64;  // tokens per chunk of a walk

// One walk (linattn_walk.h): out_t = sum_s lam^|t-s| (a_t . b_s) c_s + the
// state's part.  a, b: width K; c and out: width V.
struct WalkArgs {
  const void *a, *b, *c;     // (batch, L, Ha | Hb | Hc, K | K | V) io dtype
  const void* x;             // the gradient of g only: like c, dotted with d out / d g
  void* out;                 // (batch, L, H, V) io dtype, or float where out_f32
  const float* init;         // nullable: the state before the walk, element (v, k) of a head
                             // at v * state_sv + k * state_sk
  float* final_state;        // nullable: the state after it, (batch, H, V, K)
  float* ws;                 // the pieces' states, (pieces, batch, H, 1 or 2, V, K)
  int32_t* piece_cut;        // (pieces, batch): whether a document starts in the piece
  const float* log_decay;    // (H)
  const int32_t* seq_lens;   // nullable (batch)
  const uint8_t* reset;      // nullable (batch, L)
  const float* dlast;        // nullable: the gradient of g's last term, (batch, H, K, V)
  double* dg_part;           // (H, batch * slices * spans)
  int64_t batch, L;
  int H, Ha, Hb, Hc, K, V;
  int64_t state_sv, state_sk;
  // The walk runs in nspan spans of span_chunks chunks at once; each starts
  // from the states of the pieces before it (piece_chunks chunks each, a
  // divisor of span_chunks), which a state walk leaves in ws.
  int nspan, span_chunks, pieces, piece_chunks;
  int out_f32;
  float s_intra, s_state, s_inter;
  // set by the launch
  int nsl, nspan_run;
  uint32_t nblk;
};

// the padded row width and the columns per block of a kernel
struct Tile { int KP, VB; };
hipError_t walk_bf16(const WalkArgs& a, Tile t, bool rev, bool dg, bool state, hipStream_t stream);
hipError_t walk_f32(const WalkArgs& a, Tile t, bool rev, bool dg, bool state, hipStream_t stream);

struct Problem {
  const void *q, *k, *v;
  const float *log_decay, *h0;
  const int32_t* seq_lens;
  const uint8_t* reset;
  int64_t batch, L;
  int H, Hk, Dk, Dv;
  float scale;
  bool f32;
};
struct FwdOut { void* o; float* last_state; };
struct BwdArgs {
  const void* dout;
  const float* dlast;  // nullable
  void *dq, *dk, *dv;
  float *dlog_decay, *dh0;  // nullable
};

size_t fwd_workspace(const Problem& p);
size_t bwd_workspace(const Problem& p, bool dg);
hipError_t forward(const Problem& p, const FwdOut& o, void* workspace, hipStream_t stream);
hipError_t backward(const Problem& p, const BwdArgs& b, void* workspace, hipStream_t stream);

struct StepArgs {
  float* state;
  const void *q, *k, *v;
  const float* log_decay;
  void* o;
  int64_t batch;
  int H, Hk, Dk, Dv;
  float scale;
  bool f32;
};
hipError_t step(const StepArgs& a, hipStream_t stream);

}  // namespace linattn
}  // namespace ssm66
