// expanded_grad.cuh -- arguments of the backward pass of the expanded attention.
//
// Of a token t and a key j that it sees, in one head:
//   P  = exp(scale q_t . k_j - lse_t)      dP = dout_t . v_j
//   dS = P (dP - delta_t)                  delta_t = dout_t . out_t - dlse_t
//   dv_j = sum_t P dout_t    dk_j = scale sum_t dS q_t    dq_t = scale sum_j dS k_j
// where q and k are both parts, and the tail's gradient is that part of dk summed
// over the heads.
#pragma once

#include "expanded_attend.cuh"

namespace satk {

// Tokens of a tile whose range of row ends is kept (expanded_grad_prepare).
constexpr int kGradTokens = 64;

struct ExpandedGradArgs {
  ExpandedArgs f;      // the forward pass: its out and lse are inputs here
  float scale;
  const void *dout;
  int64_t ld_do_t, ld_do_h;
  const float *dlse;
  void *dq;
  int64_t ld_dq_t, ld_dq_h;
  void *dk;
  int64_t ld_dk_s, ld_dk_h;
  void *dtail;
  int64_t ld_dtail;
  void *dv;
  int64_t ld_dv_s, ld_dv_h;
  // workspace
  float2 *stats;       // [H, T]: lse in log2, delta
  int2 *ends;          // the smallest and largest row end of each tile of tokens
  float *tails;        // [H, S, dr]: the tail's gradient of each head
};

// Tiles of up to `size` rows that cut the requests: tile i of request r has slot
// starts[r] / size + r + i, so no count over the requests is needed; slots that
// no tile has are empty.
__host__ __device__ __forceinline__ int64_t tile_slots(int64_t n, int64_t R, int size) {
  return n / size + R + 1;
}

// The parts of the workspace in order, each a multiple of 16 bytes.
struct GradWorkspace {
  size_t stats, ends, tails, total;
};
inline GradWorkspace grad_workspace(int64_t T, int64_t S, int64_t R, int64_t H, int64_t dr) {
  const auto round = [](size_t x) { return (x + 15) & ~static_cast<size_t>(15); };
  GradWorkspace w;
  w.stats = 0;
  w.ends = w.stats + round(static_cast<size_t>(H) * T * sizeof(float2));
  w.tails = w.ends + round(static_cast<size_t>(tile_slots(T, R, kGradTokens)) * sizeof(int2));
  w.total = w.tails + round(static_cast<size_t>(H) * S * dr * sizeof(float));
  return w;
}

// Where request r's tokens and keys are: ascending starts, cut to the arrays.
struct Span {
  int begin, end;
};
__device__ __forceinline__ Span span_of(const int32_t *starts, int r, int n) {
  const int b = min(max(starts[r], 0), n);
  return {b, min(max(starts[r + 1], b), n)};
}
// The last request that starts at or before row x; -1 where no request has x.
__device__ __forceinline__ int request_of(const int32_t *starts, int R, int n, int x) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= x) lo = mid; else hi = mid;
  }
  if (R == 0) return -1;
  const Span s = span_of(starts, lo, n);
  return x >= s.begin && x < s.end ? lo : -1;
}

// P of a score: at most 1, also where scores are so large that lse has lost the
// digits behind the point.
__device__ __forceinline__ float grad_weight(float raw, float scale_log2, float lse_log2) {
  float x;
  asm("min.NaN.f32 %0, %1, 0f00000000;" : "=f"(x) : "f"(fmaf(raw, scale_log2, -lse_log2)));
  return exp2_fast(x);
}

// stats and ends; then dk, dv and the heads' tails, and dq, by the general kernels or
// (where they take the call) on the tensor cores; then the tail's sum.
int expanded_grad_prepare(const ExpandedGradArgs &a, int dtype, cudaStream_t stream);
bool expanded_grad_mma_fits(const ExpandedGradArgs &a);
int expanded_grad_mma(const ExpandedGradArgs &a, int dtype, cudaStream_t stream);
int expanded_grad_warp(const ExpandedGradArgs &a, int dtype, cudaStream_t stream);
int expanded_grad_tail(const ExpandedGradArgs &a, int dtype, cudaStream_t stream);

}  // namespace satk
