// vec_io.h -- N neighbouring io values in accesses of 16 bytes (gfx950 device code).
//
// The accesses are declared with the alignment of one value: global memory takes
// 16 bytes from any such address in one instruction, and tensors may begin, and
// rows of odd sizes do begin, anywhere.
#pragma once

#include "ssm_device.h"

namespace ssm66 {

struct __attribute__((packed, aligned(4))) Four32 { float v[4]; };
struct __attribute__((packed, aligned(4))) Two32 { float v[2]; };
struct __attribute__((packed, aligned(2))) Four16 { uint32_t w[2]; };
struct __attribute__((packed, aligned(2))) Two16 { uint32_t w; };
struct __attribute__((packed, aligned(2))) Eight16 { uint32_t w[4]; };

template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&f)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const Four32 v = ((const Four32*)p)[q];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[4 * q + k] = v.v[k];
    }
  } else if constexpr (N == 2) {
    const Two32 v = *(const Two32*)p;
    f[0] = v.v[0];
    f[1] = v.v[1];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) f[k] = p[k];
  }
}
template <int N>
__device__ __forceinline__ void load_n(const bf16_bits* p, float (&f)[N]) {
  if constexpr (N == 8) {
    const Eight16 v = *(const Eight16*)p;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(v.w[q] << 16);
      f[2 * q + 1] = __uint_as_float(v.w[q] & 0xffff0000u);
    }
  } else if constexpr (N == 4) {
    const Four16 v = *(const Four16*)p;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f[2 * q] = __uint_as_float(v.w[q] << 16);
      f[2 * q + 1] = __uint_as_float(v.w[q] & 0xffff0000u);
    }
  } else if constexpr (N == 2) {
    const uint32_t w = ((const Two16*)p)->w;
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
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
      ((Four32*)p)[q] = Four32{{f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]}};
  } else if constexpr (N == 2) {
    *(Two32*)p = Two32{{f[0], f[1]}};
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) p[k] = f[k];
  }
}
template <int N>
__device__ __forceinline__ void store_n(bf16_bits* p, const float (&f)[N]) {
  if constexpr (N == 8) {
    *(Eight16*)p = Eight16{{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                            pack_bf16x2(f[6], f[7])}};
  } else if constexpr (N == 4) {
    *(Four16*)p = Four16{{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])}};
  } else if constexpr (N == 2) {
    *(Two16*)p = Two16{pack_bf16x2(f[0], f[1])};
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) store_io(p + k, f[k]);
  }
}

// The first n of 8 values (all with n >= 8) as they lie in memory, zero behind
// them: on their way while the thread does other work.
template <typename T> struct Raw8;
template <> struct Raw8<bf16_bits> {
  Eight16 r;
  __device__ __forceinline__ void load(const bf16_bits* p, int n) {
    r = Eight16{};
    if (n >= 8) {
      r = *(const Eight16*)p;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) r.w[k / 2] |= (uint32_t)p[k] << (16 * (k % 2));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[2 * q] = __uint_as_float(r.w[q] << 16);
      f[2 * q + 1] = __uint_as_float(r.w[q] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  Four32 r[2];
  __device__ __forceinline__ void load(const float* p, int n) {
    r[0] = r[1] = Four32{};
    if (n >= 8) {
      r[0] = ((const Four32*)p)[0];
      r[1] = ((const Four32*)p)[1];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) r[k / 4].v[k % 4] = p[k];
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = r[k / 4].v[k % 4];
  }
};
// the first n of 8 values
template <typename T>
__device__ __forceinline__ void store_8(T* p, const float (&f)[8], int n) {
  if (n >= 8) {
    store_n<8>(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store_io(p + k, f[k]);
  }
}

// the value as it will be read back from memory of its type
__device__ __forceinline__ float as_stored(float v, const float*) { return v; }
__device__ __forceinline__ float as_stored(float v, const bf16_bits*) { return (float)(__bf16)v; }

}  // namespace ssm66
