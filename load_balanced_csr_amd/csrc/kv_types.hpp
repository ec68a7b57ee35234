// Element types of the paged-cache kernels: conversions between 32-bit
// floats and what caches and queries hold.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace spmv {

typedef _Float16 f16;
typedef __bf16 bf16;
struct f8 {           // e4m3: 4 exponent and 3 mantissa bits, bias 7, no infinities
  uint8_t bits;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(f16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(bf16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(f8 x) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_cvt_f32_fp8((int)x.bits, 0);
#else
  return 0.f;
#endif
}

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  return (T)x;        // round to nearest even
}
// Round to nearest even, saturating: the largest e4m3 value is 448, and what
// the conversion would turn into NaN (beyond it, and infinities) becomes
// +-448. NaN stays NaN: the comparisons are false for it.
template <>
__device__ __forceinline__ f8 from_f32<f8>(float x) {
  x = x > 448.f ? 448.f : x;
  x = x < -448.f ? -448.f : x;
#if defined(__HIP_DEVICE_COMPILE__)
  return f8{(uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff)};
#else
  return f8{0};
#endif
}

}  // namespace spmv
