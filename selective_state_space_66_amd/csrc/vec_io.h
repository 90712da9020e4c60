// vec_io.h -- N neighbouring io values in one or two 16-byte accesses, or in one
// of their own size (gfx950 device code).
#pragma once

#include "ssm_device.h"

namespace ssm66 {

template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 v = ((const float4*)p)[q];
      f[4 * q] = v.x; f[4 * q + 1] = v.y; f[4 * q + 2] = v.z; f[4 * q + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = p[k];
  }
}
template <int N>
__device__ __forceinline__ void load_n(const bf16_bits* p, float (&f)[N]) {
  if constexpr (N == 8) {
    const uint4 v = *(const uint4*)p;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(w[q] << 16);
      f[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  } else if constexpr (N == 4) {
    const uint2 v = *(const uint2*)p;
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = to_f32(p[k]);
  }
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      ((float4*)p)[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] = f[k];
  }
}
template <int N>
__device__ __forceinline__ void store_n(bf16_bits* p, const float (&f)[N]) {
  if constexpr (N == 8) {
    *(uint4*)p = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                            pack_bf16x2(f[6], f[7]));
  } else if constexpr (N == 4) {
    *(uint2*)p = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) store_io(p + k, f[k]);
  }
}

// N values as they lie in memory: on their way while the thread does other work
template <typename T, int N> struct RawN {
  T v[N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = p[k];
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = to_f32(v[k]);
  }
};
template <> struct RawN<bf16_bits, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_bits* p) { v = *(const uint4*)p; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(w[q] << 16);
      f[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
  }
};
template <> struct RawN<float, 8> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = ((const float4*)p)[0];
    v[1] = ((const float4*)p)[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = v[0].x; f[1] = v[0].y; f[2] = v[0].z; f[3] = v[0].w;
    f[4] = v[1].x; f[5] = v[1].y; f[6] = v[1].z; f[7] = v[1].w;
  }
};

// the value as it will be read back from memory of its type
__device__ __forceinline__ float as_stored(float v, const float*) { return v; }
__device__ __forceinline__ float as_stored(float v, const bf16_bits*) { return (float)(__bf16)v; }

}  // namespace ssm66
