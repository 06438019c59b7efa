// latent_merge.cu -- satk_latent_merge: W partial attention results over
// disjoint keys joined by their log-sum-exps.
//
// One thread per eight output columns of a (token, head).  Ranks go in groups of
// eight whose lse values and 16-byte parts are all asked for together; further
// groups rescale by the running maximum.  Each part is read once and the result
// written once: memory-bound.  Rows that are not 16-byte aligned take one column
// per thread.  Eight parts of 128 x 64 rows of 512 columns: 16.1 us, 4.7 TB/s.
#include "latent_common.cuh"

namespace satk {
namespace {

constexpr int kMergeBlock = 256;

struct MergeArgs {
  const void *parts;
  int W, H, dv;
  int64_t rows;  // T * H
  int64_t ld_w, ld_t, ld_h;
  const float *lse;
  void *out;
  int64_t ld_out_t, ld_out_h;
  float *lse_out;
};

template <class E, int VEC>
__global__ void __launch_bounds__(kMergeBlock) latent_merge_kernel(MergeArgs a) {
  const int per_row = (a.dv + VEC - 1) / VEC;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kMergeBlock + threadIdx.x;
  const int64_t row = i / per_row;
  if (row >= a.rows) return;
  const int c = static_cast<int>(i - row * per_row) * VEC;
  const int64_t t = row / a.H;
  const int h = static_cast<int>(row - t * a.H);
  const E *part = static_cast<const E *>(a.parts) + t * a.ld_t + h * a.ld_h + c;
  const float *lse = a.lse + row;
  constexpr int kGroup = 8;
  float ref = -INFINITY, sum = 0.f;
  float acc[VEC] = {};
  for (int w0 = 0; w0 < a.W; w0 += kGroup) {
    float x[kGroup];
    Pack8<E> v[kGroup];
    E one[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (w0 + i < a.W) {
        x[i] = __ldg(lse + (w0 + i) * a.rows);
        if constexpr (VEC == 8) v[i].u = __ldg(reinterpret_cast<const uint4 *>(part + (w0 + i) * a.ld_w));
        else one[i] = part[(w0 + i) * a.ld_w];
      } else {
        x[i] = -INFINITY;
      }
    }
    float top = ref;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) top = fmaxf(top, x[i]);
    const float base = top == -INFINITY ? 0.f : top;
    const float keep = exp2_fast((ref - base) * kLog2e);
    ref = top;
    if (w0 > 0) {
      sum *= keep;
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= keep;
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (x[i] == -INFINITY) continue;  // nothing of an empty part counts
      const float p = exp2_fast((x[i] - base) * kLog2e);
      sum += p;
      if constexpr (VEC == 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = Elem<E>::to2(v[i].h[j]);
          acc[2 * j] = fmaf(p, f.x, acc[2 * j]);
          acc[2 * j + 1] = fmaf(p, f.y, acc[2 * j + 1]);
        }
      } else {
        acc[0] = fmaf(p, Elem<E>::to(one[i]), acc[0]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h + c;
  if constexpr (VEC == 8) {
    Pack8<E> v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v.h[j] = Elem<E>::from2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
    *reinterpret_cast<uint4 *>(out) = v.u;
  } else {
    out[0] = Elem<E>::from(acc[0] * inv);
  }
  if (c == 0 && a.lse_out != nullptr) a.lse_out[row] = sum == 0.f ? -INFINITY : ref + logf(sum);
}

}  // namespace
}  // namespace satk

extern "C" int satk_latent_merge(const void *parts, int dtype, int32_t W, int64_t T, int32_t H,
                                 int32_t dv, int64_t ld_w, int64_t ld_t, int64_t ld_h,
                                 const float *lse, void *out, int64_t ld_out_t, int64_t ld_out_h,
                                 float *lse_out, satk_stream_t stream) {
  using namespace satk;
  if (parts == nullptr || lse == nullptr || out == nullptr || !is_16bit(dtype) || W < 1 || T < 0 ||
      H < 1 || dv < 1 || T > INT32_MAX || T * H > INT32_MAX || (H > 1 && (ld_h < dv || ld_out_h < dv)) ||
      (T > 1 && (ld_t < dv || ld_out_t < dv)) || (W > 1 && ld_w < dv))
    return SATK_EINVAL;
  if (W > SATK_LATENT_MAX_RANKS) return SATK_EUNSUPPORTED;
  if (T == 0) return SATK_OK;
  MergeArgs a{parts, W, H, dv, T * H, ld_w, ld_t, ld_h, lse, out, ld_out_t, ld_out_h, lse_out};
  const bool vec = aligned16(parts) && aligned16(out) && dv % 8 == 0 &&
                   (H == 1 || (ld_h % 8 == 0 && ld_out_h % 8 == 0)) &&
                   (T == 1 || (ld_t % 8 == 0 && ld_out_t % 8 == 0)) && (W == 1 || ld_w % 8 == 0);
  const int64_t threads = a.rows * (vec ? dv / 8 : dv);
  const int64_t grid = (threads + kMergeBlock - 1) / kMergeBlock;
  if (grid > INT32_MAX) return SATK_EINVAL;
  auto launch = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(grid), kMergeBlock, 0, as_stream(stream)>>>(a);
  };
  if (dtype == SATK_BF16)
    vec ? launch(latent_merge_kernel<__nv_bfloat16, 8>) : launch(latent_merge_kernel<__nv_bfloat16, 1>);
  else
    vec ? launch(latent_merge_kernel<__half, 8>) : launch(latent_merge_kernel<__half, 1>);
  return launch_status();
}
