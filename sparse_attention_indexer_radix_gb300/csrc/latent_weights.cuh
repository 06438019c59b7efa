// latent_weights.cuh -- arguments of the attention weights over selected rows.
#pragma once

#include "latent_common.cuh"

namespace satk {

struct WeightsArgs {
  const void *q;
  int T, H, D;
  int64_t ld_q_t, ld_q_h;
  const void *cache;
  int64_t cache_rows, ld_cache;
  const int32_t *rows;
  int64_t ld_rows;
  int k;
  const int32_t *counts;
  float scale;
  const float *lse;
  float *out;
  int64_t ld_out;
  int32_t *status;
};

// The row of a token's entry, or -1 for one that is skipped.
__device__ __forceinline__ int64_t entry_row(const WeightsArgs &a, int t, int j, int count) {
  if (j >= count) return -1;
  const int row = a.rows[t * a.ld_rows + j];
  if (row < 0) return -1;
  if (row >= a.cache_rows) {
    if (a.status != nullptr) atomicOr(a.status, SATK_STATUS_BAD_ROW);
    return -1;
  }
  return row;
}

__device__ __forceinline__ int entry_count(const WeightsArgs &a, int t) {
  return a.counts == nullptr ? a.k : min(max(a.counts[t], 0), a.k);
}

// One head's weight from its score and its normaliser: the difference first, so that
// only its own size is rounded on the way to log2, then at most 1 (scores of a size at
// which lse has lost the digits behind the point); nothing for a head that saw no key.
__device__ __forceinline__ float head_weight(float raw, float scale, float lse) {
  float x;
  asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(x) : "f"(fmaf(raw, scale, -lse)));
  return lse == -INFINITY ? 0.f : exp2_fast(x * kLog2e);
}

// The tensor-core kernel: whether it takes this call, and the call.
bool latent_weights_mma_fits(const WeightsArgs &a);
int latent_weights_mma(const WeightsArgs &a, int dtype, cudaStream_t stream);

// The general kernel: any widths, strides and alignment.
int latent_weights_warp(const WeightsArgs &a, int dtype, cudaStream_t stream);

}  // namespace satk
