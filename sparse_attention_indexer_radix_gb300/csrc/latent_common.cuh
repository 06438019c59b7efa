// latent_common.cuh -- element conversions and argument checks shared by the
// latent-cache operators.
#pragma once

#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "satk_device.cuh"
#include "satk_host.hpp"

namespace satk {

template <class E>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  using T2 = __nv_bfloat162;
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16(x); }
  static __device__ __forceinline__ float2 to2(T2 x) { return __bfloat1622float2(x); }
  static __device__ __forceinline__ T2 from2(float a, float b) {
    return __floats2bfloat162_rn(a, b);
  }
};
template <>
struct Elem<__half> {
  using T2 = __half2;
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half(x); }
  static __device__ __forceinline__ float2 to2(T2 x) { return __half22float2(x); }
  static __device__ __forceinline__ T2 from2(float a, float b) { return __floats2half2_rn(a, b); }
};

// Eight 16-bit elements as one 16-byte access.
template <class E>
union Pack8 {
  uint4 u;
  typename Elem<E>::T2 h[4];
};

// exp2 of x <= 0 (or the small positive range of a lagging maximum), and
// log2: the hardware approximations, relative error about 2^-22.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

inline bool is_16bit(int dtype) { return dtype == SATK_BF16 || dtype == SATK_F16; }

}  // namespace satk
