// Element types of the decoder operators: fp32, fp16, bf16 in memory, fp32 in registers.
#pragma once
#include "pi_device.hpp"

namespace pi {

typedef __bf16 bf16_t;
typedef half_t half4_t __attribute__((ext_vector_type(4)));
typedef half_t half8_t __attribute__((ext_vector_type(8)));
typedef bf16_t bf4_t __attribute__((ext_vector_type(4)));
typedef bf16_t bf8_t __attribute__((ext_vector_type(8)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// 8 consecutive elements at p (16-byte aligned) as floats. Conversions to fp32 are exact.
__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) { o[i] = a[i]; o[4 + i] = b[i]; }
}
__device__ __forceinline__ void load8(const half_t* p, float (&o)[8]) {
  const half8_t a = *reinterpret_cast<const half8_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = (float)a[i];
}
__device__ __forceinline__ void load8(const bf16_t* p, float (&o)[8]) {
  const u32x4 a = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) { o[2 * i] = u2f(a[i] << 16); o[2 * i + 1] = u2f(a[i] & 0xFFFF0000u); }
}

// 8 floats to 8 consecutive elements at p (16-byte aligned), rounded to nearest even.
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<f32x4*>(p)[0] = (f32x4){v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4*>(p)[1] = (f32x4){v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(half_t* p, const float (&v)[8]) {
  half8_t a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (half_t)v[i];
  *reinterpret_cast<half8_t*>(p) = a;
}
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  bf8_t a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (bf16_t)v[i];
  *reinterpret_cast<bf8_t*>(p) = a;
}

}  // namespace pi
