// philox.h -- counter-based random numbers (gfx950 device code).
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011): a bijection of a 128-bit counter under
// a 64-bit key, four 32-bit words a call.  A round multiplies two words by
// constants to 64 bits and mixes the halves, the key moves on by two constants.
// The published vectors are among the tests.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm66 {

// The words 4 * block .. 4 * block + 3 of the stream (seed, offset).  seed and
// offset are the same for all threads: their arithmetic stays scalar.
__device__ __forceinline__ void philox_block(uint64_t seed, uint64_t offset, uint64_t block,
                                             uint32_t (&out)[4]) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  out[0] = c0; out[1] = c1; out[2] = c2; out[3] = c3;
}

// A rate of dropping as what is compared and multiplied: a value whose word is
// under `below` becomes 0, the others are multiplied with `factor`.
struct Drop {
  const int64_t* rng;  // device: seed, offset; null where nothing is dropped
  uint64_t site;       // added to the offset
  uint32_t below;
  float factor;
};

// p in [0, 1): p 2^32 is whole for p of 2^-8 and more, rounded down below
inline Drop drop_of(float p, const int64_t* rng, int64_t site) {
  Drop d;
  d.rng = p > 0.0f ? rng : nullptr;
  d.site = (uint64_t)site;
  d.below = (uint32_t)((double)p * 4294967296.0);
  d.factor = (float)(1.0 / (1.0 - (double)p));
  return d;
}

// The factors of eight values from `at` on, a multiple of 4.
__device__ __forceinline__ void drop_factors(const Drop& d, uint64_t seed, uint64_t offset,
                                             int64_t at, float (&f)[8]) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t w[4];
    philox_block(seed, offset, ((uint64_t)at >> 2) + b, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[4 * b + k] = w[k] >= d.below ? d.factor : 0.0f;
  }
}
__device__ __forceinline__ uint32_t either(bool second, uint32_t a, uint32_t b) { return second ? b : a; }
// The same from anywhere: they lie in three blocks.
__device__ __forceinline__ void drop_factors_any(const Drop& d, uint64_t seed, uint64_t offset,
                                                 int64_t at, float (&f)[8]) {
  uint32_t w[12];
#pragma unroll
  for (int b = 0; b < 3; ++b) {
    uint32_t t[4];
    philox_block(seed, offset, ((uint64_t)at >> 2) + b, t);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[4 * b + k] = t[k];
  }
  const int s = (int)(at & 3);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t lo = either(s & 1, w[k], w[k + 1]), hi = either(s & 1, w[k + 2], w[k + 3]);
    f[k] = either(s & 2, lo, hi) >= d.below ? d.factor : 0.0f;
  }
}

// a dropped value is 0 whatever it was
__device__ __forceinline__ float dropped(float v, float f) { return f != 0.0f ? v * f : 0.0f; }

}  // namespace ssm66
