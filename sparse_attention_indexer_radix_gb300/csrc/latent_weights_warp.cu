// latent_weights_warp.cu -- attention weights over selected rows, one warp per
// (token, entry): the cache row in registers, one element of every 32 per lane,
// and a product a head.  Any width, stride and alignment; every warp reads its
// token's queries again, so it is instruction-bound.
#include "latent_weights.cuh"

namespace satk {
namespace {

constexpr int kWarps = 4;

template <class E>
__global__ void __launch_bounds__(kWarps * 32) latent_weights_warp_kernel(WeightsArgs a, int64_t n) {
  constexpr int kD = (SATK_LATENT_MAX + SATK_LATENT_TAIL_MAX) / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= n) return;
  const int t = static_cast<int>(id / a.k), j = static_cast<int>(id % a.k);
  const int64_t row = entry_row(a, t, j, entry_count(a, t));
  float sum = 0.f;
  if (row >= 0) {
    const E *key = static_cast<const E *>(a.cache) + row * a.ld_cache;
    float v[kD];
#pragma unroll
    for (int i = 0; i < kD; ++i) {
      const int c = i * 32 + lane;
      v[i] = c < a.D ? Elem<E>::to(key[c]) : 0.f;
    }
    for (int h = 0; h < a.H; ++h) {
      const E *q = static_cast<const E *>(a.q) + t * a.ld_q_t + h * a.ld_q_h;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kD; ++i) {
        const int c = i * 32 + lane;
        if (c < a.D) s = fmaf(Elem<E>::to(q[c]), v[i], s);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      sum += head_weight(s, a.scale, a.lse[static_cast<int64_t>(t) * a.H + h]);
    }
  }
  if (lane == 0) a.out[t * a.ld_out + j] = sum / a.H;
}

}  // namespace

int latent_weights_warp(const WeightsArgs &a, int dtype, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k, grid = (n + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  if (dtype == SATK_BF16)
    latent_weights_warp_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a, n);
  else
    latent_weights_warp_kernel<__half><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a, n);
  return launch_status();
}

}  // namespace satk
