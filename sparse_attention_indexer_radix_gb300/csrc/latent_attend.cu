// latent_attend.cu -- entry points of the attention over latent cache rows:
// satk_latent_attend (whole paged caches, causal ends and drafted trees) and
// satk_latent_attend_rows (selected rows).
#include "latent_attend.cuh"

namespace satk {
namespace {

// The checks both entry points share; SATK_OK when the call may go on.
int check(const LatentArgs &a, int dtype, int64_t T, int64_t dr, float scale,
          const void *workspace, size_t workspace_bytes) {
  if (a.q == nullptr || a.cache == nullptr || a.out == nullptr || workspace == nullptr ||
      !is_16bit(dtype) || T < 0 || T > INT32_MAX || a.H < 1 || a.dl < 1 || dr < 0 ||
      (T > 1 && (a.ld_q_t < a.D || a.ld_out_t < a.dl)) ||
      (a.H > 1 && (a.ld_q_h < a.D || a.ld_out_h < a.dl)) || a.ld_cache < a.D ||
      a.cache_rows < 0 || !std::isfinite(scale) || !aligned16(workspace))
    return SATK_EINVAL;
  if (a.H > 1024 || a.dl > SATK_LATENT_MAX || dr > SATK_LATENT_TAIL_MAX) return SATK_EUNSUPPORTED;
  if (workspace_bytes < satk_latent_workspace_bytes(a.H, a.dl)) return SATK_EINVAL;
  return SATK_OK;
}

int dispatch(const LatentArgs &a, int dtype, int tokens_per_request, void *workspace,
             cudaStream_t stream) {
  if (latent_attend_mma_fits(a))
    return latent_attend_mma(a, dtype, tokens_per_request, workspace, stream);
  return latent_attend_warp(a, dtype, stream);
}

}  // namespace
}  // namespace satk

extern "C" size_t satk_latent_workspace_bytes(int32_t H, int32_t dl) {
  if (H < 1 || H > 1024 || dl < 1 || dl > SATK_LATENT_MAX) return 0;
  return satk::latent_attend_mma_workspace(H, dl);
}

extern "C" int satk_latent_attend(const void *q, int dtype, int64_t T, int32_t H, int32_t dl,
                                  int32_t dr, int64_t ld_q_t, int64_t ld_q_h, const void *cache,
                                  int64_t cache_rows, int64_t ld_cache, const int32_t *req_id,
                                  const int32_t *block_table, int64_t table_rows,
                                  int64_t ld_block_table, int32_t max_blocks, int32_t block_size,
                                  int64_t stride_rows, const int32_t *row_ends,
                                  const int32_t *tree, int32_t tree_words, float scale, void *out,
                                  int64_t ld_out_t, int64_t ld_out_h, float *lse, void *workspace,
                                  size_t workspace_bytes, int32_t *status, satk_stream_t stream) {
  using namespace satk;
  if (req_id == nullptr || block_table == nullptr || row_ends == nullptr || table_rows < 0 ||
      max_blocks < 0 || ld_block_table < max_blocks || block_size < 1 || stride_rows < 0 ||
      (tree != nullptr && tree_words < 1) || dl < 1 || dr < 0)
    return SATK_EINVAL;
  if (dl > SATK_LATENT_MAX || dr > SATK_LATENT_TAIL_MAX || (tree != nullptr && tree_words > 32))
    return SATK_EUNSUPPORTED;
  const int64_t reach = static_cast<int64_t>(max_blocks) * block_size;
  // keys stay below 2**31 - 2048 so that key indices and tile ends fit int32
  const int max_keys = static_cast<int>(reach < INT32_MAX - 2048 ? reach : INT32_MAX - 2048);
  LatentArgs a{q,          static_cast<int>(T), H,      dl,        dl + dr,    ld_q_t,
               ld_q_h,     cache,      cache_rows, ld_cache,  req_id,     block_table,
               table_rows, ld_block_table, max_keys, block_size, log2_or(block_size), stride_rows,
               row_ends,   tree,       tree_words, nullptr,   nullptr,    0,
               0,          scale * kLog2e, out,    ld_out_t,  ld_out_h,   lse,
               status};
  const int rc = check(a, dtype, T, dr, scale, workspace, workspace_bytes);
  if (rc != SATK_OK || T == 0) return rc;
  const int64_t per = table_rows > 0 ? (T + table_rows - 1) / table_rows : 1;
  return dispatch(a, dtype, static_cast<int>(per), workspace, as_stream(stream));
}

extern "C" int satk_latent_attend_rows(const void *q, int dtype, int64_t T, int32_t H, int32_t dl,
                                       int32_t dr, int64_t ld_q_t, int64_t ld_q_h,
                                       const void *cache, int64_t cache_rows, int64_t ld_cache,
                                       const int32_t *rows, int64_t ld_rows, int32_t k,
                                       const int32_t *counts, float scale, void *out,
                                       int64_t ld_out_t, int64_t ld_out_h, float *lse,
                                       void *workspace, size_t workspace_bytes, int32_t *status,
                                       satk_stream_t stream) {
  using namespace satk;
  if (rows == nullptr || k < 1 || k > INT32_MAX - 2048 || (T > 1 && ld_rows < k) || dl < 1 ||
      dr < 0)
    return SATK_EINVAL;
  if (dl > SATK_LATENT_MAX || dr > SATK_LATENT_TAIL_MAX) return SATK_EUNSUPPORTED;
  LatentArgs a{q,       static_cast<int>(T), H,  dl,      dl + dr,  ld_q_t,
               ld_q_h,  cache,   cache_rows, ld_cache, nullptr, nullptr,
               0,       0,       0,          1,        0,       0,
               nullptr, nullptr, 0,          rows,     counts,  ld_rows,
               k,       scale * kLog2e, out, ld_out_t, ld_out_h, lse,
               status};
  const int rc = check(a, dtype, T, dr, scale, workspace, workspace_bytes);
  if (rc != SATK_OK || T == 0) return rc;
  return dispatch(a, dtype, 1, workspace, as_stream(stream));
}
