// dropout.hip -- dropout whose mask is computed from a counter and never stored.
//
//   y_e = (word_e >= p 2^32 ? x_e / (1 - p) : 0) + residual_e,
// word_e the e-th word of the generator's stream (philox.h).  The gradient of x
// is the same map of dy without the residual.
//
// A thread takes eight values: two calls of the generator and one or two 16-byte
// accesses a tensor.  HBM bounds it: 16384 x 1536, bf16, with a residual 26 us (151
// MB, 5.8 TB/s, part of it from the Infinity Cache); its 27 vector instructions a
// value, most of them the generator's, would take 17.  Tensors off a 16-byte boundary, and the last values, take
// the same values one at a time.
#include "dropout_launch.h"
#include "vec_io.h"

namespace ssm66 {
namespace dropout {

namespace {

constexpr int kVec = 8;

template <typename T, typename TY, bool WIDE>
__global__ __launch_bounds__(256) void dropout_kernel(const Args p) {
  const T* const x = (const T*)p.x;
  const TY* const res = (const TY*)p.residual;
  TY* const y = (TY*)p.y;
  uint64_t seed = 0, offset = 0;
  if (p.drop.rng) {
    seed = (uint64_t)p.drop.rng[0];
    offset = (uint64_t)p.drop.rng[1] + p.drop.site;
  }
  const int64_t step = (int64_t)gridDim.x * 256 * kVec;
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kVec; at < p.n; at += step) {
    const int here = p.n - at < kVec ? (int)(p.n - at) : kVec;
    float v[kVec], r[kVec], f[kVec];
    if (WIDE && here == kVec) {
      load_n<kVec>(x + at, v);
      if (res) load_n<kVec>(res + at, r);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        v[k] = k < here ? to_f32(x[at + k]) : 0.0f;
        r[k] = k < here && res ? to_f32(res[at + k]) : 0.0f;
      }
    }
    if (p.drop.rng) {
      drop_factors<kVec>(p.drop, seed, offset, at, f);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = dropped(v[k], f[k]);
    }
    if (res)
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] += r[k];
    if (WIDE && here == kVec) {
      store_n<kVec>(y + at, v);
    } else {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k < here) store_io(y + at + k, v[k]);
    }
  }
}

template <typename T, typename TY>
hipError_t launch(const Args& p, hipStream_t s) {
  const bool wide = (((uintptr_t)p.x | (uintptr_t)p.residual | (uintptr_t)p.y) & 15) == 0;
  const int64_t blocks = (p.n + 256 * kVec - 1) / (256 * kVec);
  const unsigned g = (unsigned)(blocks < 65536 ? blocks : 65536);
  if (wide) dropout_kernel<T, TY, true><<<g, 256, 0, s>>>(p);
  else dropout_kernel<T, TY, false><<<g, 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t run(const Args& p, bool x_f32, bool y_f32, hipStream_t s) {
  if (x_f32) return y_f32 ? launch<float, float>(p, s) : launch<float, bf16_bits>(p, s);
  return y_f32 ? launch<bf16_bits, float>(p, s) : launch<bf16_bits, bf16_bits>(p, s);
}

}  // namespace dropout
}  // namespace ssm66
