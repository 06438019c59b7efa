// latent_attend_warp.cu -- attention over latent cache rows, one warp per
// (token, head).
//
// softmax(scale q . k_j) k_j[:dl] in one pass over the keys a token sees: the
// warp holds its query and its fp32 accumulator in registers (one element of
// every 32 per lane), takes a key's dot product by a warp reduction and keeps
// the running maximum and sum.  Every element is its own 2-byte access, so any
// width, stride and alignment works; each key row is read again by every
// head's warp, which makes it L2- and instruction-bound.  It serves what the
// tensor-core kernel's 16-byte loads do not fit (widths or row strides that are
// not multiples of eight, unaligned caches): 64 requests x up to 16384 keys x 32
// heads take 23.8 ms here and 0.11 ms there.
#include "latent_attend.cuh"

namespace satk {
namespace {

constexpr int kWarps = 4;

template <class E>
__global__ void __launch_bounds__(kWarps * 32) latent_attend_warp_kernel(LatentArgs a) {
  constexpr int kQ = (SATK_LATENT_MAX + SATK_LATENT_TAIL_MAX) / 32, kV = SATK_LATENT_MAX / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(a.T) * a.H) return;
  const int t = static_cast<int>(id / a.H), h = static_cast<int>(id % a.H);
  const E *q = static_cast<const E *>(a.q) + t * a.ld_q_t + h * a.ld_q_h;
  float qv[kQ], acc[kV];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int c = i * 32 + lane;
    qv[i] = c < a.D ? Elem<E>::to(q[c]) * a.scale_log2 : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  const int end = token_end(a, t), extent = token_extent(a, t, end);
  const int r = a.rows == nullptr ? a.req_id[t] : 0;
  const int first = a.rows == nullptr ? max(a.row_ends[t], 0) : 0;
  float m = -INFINITY, l = 0.f;
  for (int j0 = 0; j0 < extent; j0 += 32) {
    const int j = j0 + lane;
    int64_t mine = -1;
    if (j < end || (j < extent && tree_bit(a, t, j - first))) mine = key_row(a, t, r, j);
    unsigned live = __ballot_sync(~0u, mine >= 0);
    while (live != 0) {
      const int src = __ffs(live) - 1;
      live &= live - 1;
      const E *key = static_cast<const E *>(a.cache) + __shfl_sync(~0u, mine, src) * a.ld_cache;
      float kv[kQ], s = 0.f;
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        const int c = i * 32 + lane;
        kv[i] = c < a.D ? Elem<E>::to(key[c]) : 0.f;
        s = fmaf(qv[i], kv[i], s);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
      if (s > m) {
        const float f = exp2_fast(m - s);
        m = s;
        l *= f;
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] *= f;
      }
      const float p = exp2_fast(s - (m == -INFINITY ? 0.f : m));
      l += p;
#pragma unroll
      for (int i = 0; i < kV; ++i) acc[i] = fmaf(p, kv[i], acc[i]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = i * 32 + lane;
    if (c < a.dl) out[c] = Elem<E>::from(acc[i] * inv);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[id] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

int latent_attend_warp(const LatentArgs &a, int dtype, cudaStream_t stream) {
  const int64_t grid = (static_cast<int64_t>(a.T) * a.H + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  if (dtype == SATK_BF16)
    latent_attend_warp_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  else
    latent_attend_warp_kernel<__half><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  return launch_status();
}

}  // namespace satk
