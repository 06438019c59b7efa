// expanded_attend.cu -- entry point satk_latent_attend_expanded.
#include "expanded_attend.cuh"

extern "C" int satk_latent_attend_expanded(const void *q, int dtype, int64_t T, int32_t H,
                                           int32_t dn, int32_t dr, int64_t ld_q_t, int64_t ld_q_h,
                                           const void *k, int64_t S, int64_t ld_k_s,
                                           int64_t ld_k_h, const void *tail, int64_t ld_tail,
                                           const void *v, int32_t dv, int64_t ld_v_s,
                                           int64_t ld_v_h, const int32_t *token_starts,
                                           const int32_t *key_starts, int32_t R,
                                           const int32_t *row_ends, float scale, void *out,
                                           int64_t ld_out_t, int64_t ld_out_h, float *lse,
                                           satk_stream_t stream) {
  using namespace satk;
  if (q == nullptr || k == nullptr || v == nullptr || token_starts == nullptr ||
      key_starts == nullptr || row_ends == nullptr || out == nullptr ||
      (tail == nullptr && dr > 0) || !is_16bit(dtype) || T < 0 || T > INT32_MAX || S < 0 ||
      S > INT32_MAX || R < 0 || H < 1 || dn < 1 || dr < 0 || dv < 1 || !std::isfinite(scale))
    return SATK_EINVAL;
  if (H > 1024 || static_cast<int64_t>(dn) + dr > SATK_EXPANDED_MAX_QK || dv > SATK_EXPANDED_MAX_V)
    return SATK_EUNSUPPORTED;
  if ((T > 1 && (ld_q_t < dn + dr || ld_out_t < dv)) || (H > 1 && (ld_q_h < dn + dr || ld_out_h < dv)) ||
      (S > 1 && (ld_k_s < dn || ld_v_s < dv || ld_tail < dr)) || (H > 1 && (ld_k_h < dn || ld_v_h < dv)))
    return SATK_EINVAL;
  if (T == 0) return SATK_OK;
  ExpandedArgs a{q,    static_cast<int>(T), H,      dn,           dr,         dv,   ld_q_t, ld_q_h,
                 k,    static_cast<int>(S), ld_k_s, ld_k_h,       tail,       ld_tail, v,   ld_v_s,
                 ld_v_h, token_starts,      key_starts, R,        row_ends,   scale * kLog2e,
                 out,  ld_out_t,            ld_out_h, lse};
  if (expanded_attend_mma_fits(a)) return expanded_attend_mma(a, dtype, as_stream(stream));
  return expanded_attend_warp(a, dtype, as_stream(stream));
}
