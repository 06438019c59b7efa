// expanded_attend.cuh -- arguments of the expanded (per-head) attention.
#pragma once

#include "latent_common.cuh"

namespace satk {

struct ExpandedArgs {
  const void *q;
  int T, H, dn, dr, dv;
  int64_t ld_q_t, ld_q_h;
  const void *k;
  int S;
  int64_t ld_k_s, ld_k_h;
  const void *tail;
  int64_t ld_tail;
  const void *v;
  int64_t ld_v_s, ld_v_h;
  const int32_t *token_starts, *key_starts;
  int R;
  const int32_t *row_ends;
  float scale_log2;
  void *out;
  int64_t ld_out_t, ld_out_h;
  float *lse;
};

// The general kernel: any widths, strides and alignment.
int expanded_attend_warp(const ExpandedArgs &a, int dtype, cudaStream_t stream);

// The tensor-core kernel (expanded_attend_mma.cu): whether it takes this call,
// and the call.
bool expanded_attend_mma_fits(const ExpandedArgs &a);
int expanded_attend_mma(const ExpandedArgs &a, int dtype, cudaStream_t stream);

}  // namespace satk
