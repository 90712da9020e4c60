// gated_scan_launch.h -- internal interface of the gated linear recurrence.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm66 {
namespace gated_scan {

constexpr int kKeep = 64;  // tokens from one kept state to the next

struct Args {
  const void *x, *r, *i;     // (batch, L, dim) io dtype
  const float* decay;        // (dim)
  const float* h0;           // nullable (batch, dim)
  const int32_t* seq_lens;   // nullable (batch)
  const uint8_t* reset;      // nullable (batch, L)
  int64_t batch, L;
  int dim;
  // forwards
  void* y;
  float* last_state;         // nullable (batch, dim)
  float* states;             // (batch, kept, dim): the state before every kKeep tokens; nullable forwards
  // backwards
  const void* dy;
  const float* dlast;        // nullable (batch, dim)
  void *dx, *dr, *di;
  float* ddecay;             // nullable (dim)
  float* dh0;                // nullable (batch, dim)
  void* ws;
  // set by the launch
  uint32_t* tickets;         // one counter in 128 bytes
  uint64_t *sums, *groups;   // (chunks, batch, dim), (groups of chunks, batch, dim)
  float* part;               // (chunks * batch, dim)
  int chunks, kept, tiles;
  int group;                 // chunks from one published state to the next, a power of two
  uint32_t rows;             // batch * tiles
  uint32_t counters, blocks;
};

// whether the grid these sizes need exists
bool fits(int64_t batch, int64_t L, int64_t dim);
size_t workspace_bytes(int64_t batch, int64_t L, int64_t dim, bool backward, bool need_ddecay);
hipError_t forward(const Args& p, bool f32, hipStream_t s);
hipError_t backward(const Args& p, bool f32, hipStream_t s);

struct StepArgs {
  float* state;
  const void *x, *r, *i;
  const float* decay;
  void* y;
  int64_t batch;
  int dim;
};
hipError_t step(const StepArgs& p, bool f32, hipStream_t s);

}  // namespace gated_scan
}  // namespace ssm66
