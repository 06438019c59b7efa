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

// References of a softmax in log2.  kUnset is that of a row without a score yet:
// no finite score is below it.  A weight's exponent raw * scale - ref is one fmaf
// while the reference is at most kFine: the reference is a rounded product, so
// the fmaf is off from 0 at the largest score by that rounding, 2^-4 at kFine.
// Beyond, where the rounding grows without bound (2^76 at 1e30: a weight of
// infinity or of nothing), the product is rounded likewise before the subtraction.
constexpr float kUnset = -3.402823466e38f;
constexpr float kFine = 1048576.f;  // 2^20
__device__ __forceinline__ float far_exponent(float raw, float scale, float ref) {
  return __fsub_rn(__fmul_rn(raw, scale), ref);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Rows of 16-byte chunks; strides of dimensions of one are free.
inline bool rows_of_16_bytes(const void *p, int64_t n, int64_t ld, int64_t H, int64_t ld_h) {
  return aligned16(p) && (n <= 1 || ld % 8 == 0) && (H <= 1 || ld_h % 8 == 0);
}

inline bool is_16bit(int dtype) { return dtype == SATK_BF16 || dtype == SATK_F16; }

}  // namespace satk
