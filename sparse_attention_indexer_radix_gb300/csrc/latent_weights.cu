// latent_weights.cu -- entry point satk_latent_rows_weights.
#include "latent_weights.cuh"

extern "C" int satk_latent_rows_weights(const void *q, int dtype, int64_t T, int32_t H, int32_t D,
                                        int64_t ld_q_t, int64_t ld_q_h, const void *cache,
                                        int64_t cache_rows, int64_t ld_cache, const int32_t *rows,
                                        int64_t ld_rows, int32_t k, const int32_t *counts,
                                        float scale, const float *lse, float *out, int64_t ld_out,
                                        int32_t *status, satk_stream_t stream) {
  using namespace satk;
  if (q == nullptr || cache == nullptr || rows == nullptr || lse == nullptr || out == nullptr ||
      !is_16bit(dtype) || T < 0 || T > INT32_MAX || H < 1 || D < 1 || k < 1 || cache_rows < 0 ||
      !std::isfinite(scale))
    return SATK_EINVAL;
  if ((T > 1 && (ld_q_t < D || ld_rows < k || ld_out < k)) || (H > 1 && ld_q_h < D) ||
      (cache_rows > 1 && ld_cache < D))
    return SATK_EINVAL;
  if (H > 1024 || D > SATK_LATENT_MAX + SATK_LATENT_TAIL_MAX) return SATK_EUNSUPPORTED;
  if (T == 0) return SATK_OK;
  const WeightsArgs a{q,    static_cast<int>(T), H, D,      ld_q_t,         ld_q_h, cache, cache_rows,
                      ld_cache, rows,            ld_rows, k, counts, scale, lse,    out,
                      ld_out,   status};
  if (latent_weights_mma_fits(a)) return latent_weights_mma(a, dtype, as_stream(stream));
  return latent_weights_warp(a, dtype, as_stream(stream));
}
