// dropout.hip -- dropout whose mask is computed from a counter and never stored.
//
//   y_e = (word_e >= p 2^32 ? x_e / (1 - p) : 0) + residual_e,
// word_e the e-th word of the generator's stream (philox.h).  The gradient of x
// is the same map of dy without the residual.
//
// A thread takes eight values: two calls of the generator and one or two 16-byte
// accesses a tensor (the last values one at a time).  HBM bounds it: 16384 x 1536, bf16, with a residual 26 us (151
// MB, 5.8 TB/s, part of it from the Infinity Cache); its 27 vector instructions a
// value, most of them the generator's, would take 17.
#include "dropout_launch.h"
#include "vec_io.h"

namespace ssm66 {
namespace dropout {

namespace {

constexpr int kVec = 8;

template <typename T, typename TY>
__global__ __launch_bounds__(256) void dropout_kernel(const Args p) {
  const TY* const res = (const TY*)p.residual;
  uint64_t seed = 0, offset = 0;
  if (p.drop.rng) {
    seed = (uint64_t)p.drop.rng[0];
    offset = (uint64_t)p.drop.rng[1] + p.drop.site;
  }
  const int64_t step = (int64_t)gridDim.x * 256 * kVec;
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kVec; at < p.n; at += step) {
    const int here = p.n - at < kVec ? (int)(p.n - at) : kVec;
    Raw8<T> rx;
    Raw8<TY> rr = {};
    rx.load((const T*)p.x + at, here);
    if (res) rr.load(res + at, here);
    float v[kVec], r[kVec];
    rx.get(v);
    rr.get(r);
    if (p.drop.rng) {
      float f[kVec];
      drop_factors(p.drop, seed, offset, at, f);
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] = dropped(v[k], f[k]);
    }
    if (res)
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[k] += r[k];
    store_8((TY*)p.y + at, v, here);
  }
}

template <typename T, typename TY>
hipError_t launch(const Args& p, hipStream_t s) {
  const int64_t blocks = (p.n + 256 * kVec - 1) / (256 * kVec);
  dropout_kernel<T, TY><<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t run(const Args& p, bool x_f32, bool y_f32, hipStream_t s) {
  if (x_f32) return y_f32 ? launch<float, float>(p, s) : launch<float, bf16_bits>(p, s);
  return y_f32 ? launch<bf16_bits, float>(p, s) : launch<bf16_bits, bf16_bits>(p, s);
}

}  // namespace dropout
}  // namespace ssm66
