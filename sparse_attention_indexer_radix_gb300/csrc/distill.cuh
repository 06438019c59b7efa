// distill.cuh -- arguments and shared pieces of the distillation kernels: rows
// of student scores, each with a short list of a teacher's entries.
//
// With tau the temperature, s_v the row's scores, (id_e, x_e) its entries:
//   p_e   the teacher's share: softmax(x / tau), x / sum x or x itself
//   q_v   the student's softmax(s / tau), over the visible columns of the row or
//         over the entries
//   loss  sum_e p_e (log p_e - log q_{id_e})
//   ds_v  dloss / tau (q_v sum_e p_e - sum_{e: id_e = v} p_e)
#pragma once

#include "latent_common.cuh"

namespace satk {

constexpr int kDistillThreads = 256;

struct DistillArgs {
  const void *logits;
  int64_t rows, cols, ld;
  const int32_t *ends;
  const int32_t *ids;
  int64_t ld_ids;
  const void *teacher;
  int64_t ld_teacher;
  int k, teacher_dtype, kind;
  float inv_tau, c;  // 1 / tau; the same in units of log2
  float *loss, *lse;
  // the gradient alone
  const float *lse_in, *dloss;
  int dloss_step;    // 1, or 0: one value for every row
  void *grad;
  int64_t ld_grad;
  int chunk, chunks; // columns of a CTA, CTAs of a row
};

template <>
struct Elem<float> {
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
};

// The elements of 16 bytes as floats, and back.
template <class E>
struct Vec16 {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void to(const uint4 &u, float2 *f) {
    Pack8<E> p;
    p.u = u;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = Elem<E>::to2(p.h[i]);
  }
  static __device__ __forceinline__ uint4 from(const float2 *f) {
    Pack8<E> p;
#pragma unroll
    for (int i = 0; i < 4; ++i) p.h[i] = Elem<E>::from2(f[i].x, f[i].y);
    return p.u;
  }
};
template <>
struct Vec16<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void to(const uint4 &u, float2 *f) {
    f[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    f[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 from(const float2 *f) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
  }
};

// Two values of every thread of the CTA reduced at once: the larger ones, or the
// sums (in one order whatever runs first).
template <bool MAX>
__device__ __forceinline__ float2 block_reduce2(float2 x, float2 *at) {
  constexpr int kWarps = kDistillThreads / 32;
  auto join = [](float2 a, float2 b) {
    return MAX ? make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)) : make_float2(a.x + b.x, a.y + b.y);
  };
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    x = join(x, make_float2(__shfl_xor_sync(~0u, x.x, d), __shfl_xor_sync(~0u, x.y, d)));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = x;
  __syncthreads();
  x = at[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) x = join(x, at[w]);
  return x;
}

// An entry's value; as a weight or probability no less than 0, and NaN if it is not
// finite (infinite logits make NaN of themselves).
__device__ __forceinline__ float teacher_value(const DistillArgs &a, int64_t at) {
  float x;
  if (a.teacher_dtype == SATK_F32) x = static_cast<const float *>(a.teacher)[at];
  else if (a.teacher_dtype == SATK_BF16)
    x = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.teacher)[at]);
  else x = __half2float(static_cast<const __half *>(a.teacher)[at]);
  if (a.kind == SATK_TEACHER_LOGITS) return x;
  return x < 0.f ? 0.f : x == INFINITY ? NAN : x;
}

// The visible columns of a row.
__device__ __forceinline__ int row_end(const DistillArgs &a, int64_t row) {
  const int cols = static_cast<int>(a.cols);
  return a.ends == nullptr ? cols : min(max(a.ends[row], 0), cols);
}

// A power of two that brings a list's largest weight near 1 (from 0 or a number below
// 2^-126 it is 2^126): sums of scaled weights, and the inverses of those, are numbers
// of 32 bits whatever the weights' size, and their shares keep their bits.
__device__ __forceinline__ float list_scale(float most) {
  const int e = 254 - static_cast<int>(__float_as_uint(most) >> 23);
  return __uint_as_float(static_cast<uint32_t>(min(max(e, 1), 253)) << 23);
}

// A thread's share of a row's entries: entry i * threads + threadIdx.x for each
// i.  id is -1 for one that does not count; x is the teacher's value.
template <int PER>
struct Entries {
  int id[PER];
  float x[PER];
  __device__ __forceinline__ void load(const DistillArgs &a, int64_t row, int end) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * kDistillThreads + threadIdx.x;
      id[i] = -1;
      x[i] = a.kind == SATK_TEACHER_LOGITS ? -INFINITY : 0.f;
      if (e < a.k) {
        const int v = a.ids[row * a.ld_ids + e];
        if (v >= 0 && v < end) {
          id[i] = v;
          x[i] = teacher_value(a, row * a.ld_teacher + e);
        }
      }
    }
  }
};

}  // namespace satk
