// expanded_grad.cu -- the backward pass of the expanded attention: entry points,
// the rows' statistics before it and the tail's sum over the heads after it.
#include "expanded_grad.cuh"

namespace satk {
namespace {

constexpr int kWarps = 8;

// A warp a token and head: delta, and the normaliser in log2, head by head side by
// side (what the tiles read).  A token whose lse is -inf saw nothing: its row end
// counts as 0 wherever this is read, so a NaN of its own cannot get out.
template <class E>
__global__ void __launch_bounds__(kWarps * 32) grad_stats_kernel(ExpandedGradArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(a.f.T) * a.f.H) return;
  const int64_t t = id / a.f.H;
  const int h = static_cast<int>(id % a.f.H);
  const E *dout = static_cast<const E *>(a.dout) + t * a.ld_do_t + h * a.ld_do_h;
  const E *out = static_cast<const E *>(a.f.out) + t * a.f.ld_out_t + h * a.f.ld_out_h;
  float sum = 0.f;
  for (int c = lane; c < a.f.dv; c += 32)
    sum = fmaf(Elem<E>::to(dout[c]), Elem<E>::to(out[c]), sum);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  if (lane == 0)
    a.stats[static_cast<int64_t>(h) * a.f.T + t] =
        make_float2(a.f.lse[id] * kLog2e, sum - (a.dlse != nullptr ? a.dlse[id] : 0.f));
}

// The range of row ends of each tile of tokens, ends cut to the request's keys.
__global__ void __launch_bounds__(kWarps * 32) grad_ends_kernel(ExpandedGradArgs a, int slots) {
  const int lane = threadIdx.x & 31;
  const int slot = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (slot >= slots) return;
  int lo = 0, hi = a.f.R;  // the last request whose first slot is at or before this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (span_of(a.f.token_starts, mid, a.f.T).begin / kGradTokens + mid <= slot) lo = mid; else hi = mid;
  }
  int least = INT32_MAX, most = 0;
  if (a.f.R > 0) {
    const Span tokens = span_of(a.f.token_starts, lo, a.f.T), keys = span_of(a.f.key_starts, lo, a.f.S);
    const int64_t first = tokens.begin + static_cast<int64_t>(slot - tokens.begin / kGradTokens - lo) * kGradTokens;
    for (int64_t t = first + lane; t < first + kGradTokens; t += 32) {
      const int end = t >= tokens.begin && t < tokens.end ? min(max(a.f.row_ends[t], 0), keys.end - keys.begin) : 0;
      least = min(least, end);
      most = max(most, end);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    least = min(least, __shfl_xor_sync(~0u, least, d));
    most = max(most, __shfl_xor_sync(~0u, most, d));
  }
  if (lane == 0) a.ends[slot] = make_int2(least, most);
}

// The heads' tails in one order.
template <class E>
__global__ void __launch_bounds__(256) grad_tail_kernel(ExpandedGradArgs a, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float sum = 0.f;
  for (int h = 0; h < a.f.H; ++h) sum += a.tails[h * n + i];
  static_cast<E *>(a.dtail)[i / a.f.dr * a.ld_dtail + i % a.f.dr] = Elem<E>::from(sum);
}

}  // namespace

int expanded_grad_prepare(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  const int64_t grid = (static_cast<int64_t>(a.f.T) * a.f.H + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  if (grid > 0) {
    if (dtype == SATK_BF16)
      grad_stats_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
    else
      grad_stats_kernel<__half><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  }
  const int slots = static_cast<int>(tile_slots(a.f.T, a.f.R, kGradTokens));
  grad_ends_kernel<<<(slots + kWarps - 1) / kWarps, kWarps * 32, 0, stream>>>(a, slots);
  return launch_status();
}

int expanded_grad_tail(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.f.S) * a.f.dr, grid = (n + 255) / 256;
  if (n == 0) return SATK_OK;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  if (dtype == SATK_BF16)
    grad_tail_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a, n);
  else
    grad_tail_kernel<__half><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a, n);
  return launch_status();
}

}  // namespace satk

extern "C" size_t satk_latent_expanded_grad_workspace_bytes(int64_t T, int64_t S, int32_t R,
                                                            int32_t H, int32_t dr) {
  if (T < 0 || T > INT32_MAX || S < 0 || S > INT32_MAX || R < 0 || H < 1 || H > 1024 || dr < 0 ||
      dr > SATK_EXPANDED_MAX_QK)
    return 0;
  return satk::grad_workspace(T, S, R, H, dr).total;
}

extern "C" int satk_latent_attend_expanded_grad(
    const void *dout, int64_t ld_do_t, int64_t ld_do_h, const float *dlse, const void *q, int dtype,
    int64_t T, int32_t H, int32_t dn, int32_t dr, int64_t ld_q_t, int64_t ld_q_h, const void *k,
    int64_t S, int64_t ld_k_s, int64_t ld_k_h, const void *tail, int64_t ld_tail, const void *v,
    int32_t dv, int64_t ld_v_s, int64_t ld_v_h, const int32_t *token_starts,
    const int32_t *key_starts, int32_t R, const int32_t *row_ends, float scale, const void *out,
    int64_t ld_out_t, int64_t ld_out_h, const float *lse, void *grad_q, int64_t ld_gq_t,
    int64_t ld_gq_h, void *grad_k, int64_t ld_gk_s, int64_t ld_gk_h, void *grad_tail,
    int64_t ld_gtail, void *grad_v, int64_t ld_gv_s, int64_t ld_gv_h, void *workspace,
    size_t workspace_bytes, satk_stream_t stream) {
  using namespace satk;
  if (dout == nullptr || q == nullptr || k == nullptr || v == nullptr || token_starts == nullptr ||
      key_starts == nullptr || row_ends == nullptr || out == nullptr || lse == nullptr ||
      grad_q == nullptr || grad_k == nullptr || grad_v == nullptr || workspace == nullptr ||
      ((tail == nullptr || grad_tail == nullptr) && dr > 0) || !is_16bit(dtype) || T < 0 ||
      T > INT32_MAX || S < 0 || S > INT32_MAX || R < 0 || H < 1 || dn < 1 || dr < 0 || dv < 1 ||
      !std::isfinite(scale) || !aligned16(workspace))
    return SATK_EINVAL;
  if (H > 1024 || static_cast<int64_t>(dn) + dr > SATK_EXPANDED_MAX_QK || dv > SATK_EXPANDED_MAX_V)
    return SATK_EUNSUPPORTED;
  const int D = dn + dr;
  if ((T > 1 && (ld_q_t < D || ld_gq_t < D || ld_out_t < dv || ld_do_t < dv)) ||
      (H > 1 && (ld_q_h < D || ld_gq_h < D || ld_out_h < dv || ld_do_h < dv || ld_k_h < dn ||
                 ld_gk_h < dn || ld_v_h < dv || ld_gv_h < dv)) ||
      (S > 1 && (ld_k_s < dn || ld_gk_s < dn || ld_v_s < dv || ld_gv_s < dv || ld_tail < dr ||
                 ld_gtail < dr)))
    return SATK_EINVAL;
  const GradWorkspace w = grad_workspace(T, S, R, H, dr);
  if (workspace_bytes < w.total) return SATK_EINVAL;
  if (T == 0 && S == 0) return SATK_OK;
  char *const at = static_cast<char *>(workspace);
  ExpandedGradArgs a;
  a.f = ExpandedArgs{q,      static_cast<int>(T), H,      dn,     dr,      dv,     ld_q_t, ld_q_h,
                     k,      static_cast<int>(S), ld_k_s, ld_k_h, tail,    ld_tail, v,     ld_v_s,
                     ld_v_h, token_starts,        key_starts, R,  row_ends, scale * kLog2e,
                     const_cast<void *>(out), ld_out_t, ld_out_h, const_cast<float *>(lse)};
  a.scale = scale;
  a.dout = dout, a.ld_do_t = ld_do_t, a.ld_do_h = ld_do_h, a.dlse = dlse;
  a.dq = grad_q, a.ld_dq_t = ld_gq_t, a.ld_dq_h = ld_gq_h;
  a.dk = grad_k, a.ld_dk_s = ld_gk_s, a.ld_dk_h = ld_gk_h;
  a.dtail = grad_tail, a.ld_dtail = ld_gtail;
  a.dv = grad_v, a.ld_dv_s = ld_gv_s, a.ld_dv_h = ld_gv_h;
  a.stats = reinterpret_cast<float2 *>(at + w.stats);
  a.ends = reinterpret_cast<int2 *>(at + w.ends);
  a.tails = reinterpret_cast<float *>(at + w.tails);
  const cudaStream_t s = as_stream(stream);
  int rc = expanded_grad_prepare(a, dtype, s);
  if (rc == SATK_OK)
    rc = expanded_grad_mma_fits(a) ? expanded_grad_mma(a, dtype, s) : expanded_grad_warp(a, dtype, s);
  if (rc == SATK_OK) rc = expanded_grad_tail(a, dtype, s);
  return rc;
}
