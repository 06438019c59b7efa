// expanded_attend_warp.cu -- expanded attention, one warp per (token, head):
// one pass over the token's visible keys with the running maximum and sum,
// query and accumulator in registers, one element of every 32 per lane.  Any
// width, stride and alignment; every warp reads its keys again, so it is L2-
// and instruction-bound.  It serves widths that are not multiples of 16, rows
// that are not 16-byte aligned and scales that are not positive: 4096 tokens x
// 8192 keys x 16 heads take 104 ms here and 0.19 ms on the tensor cores.
#include "expanded_attend.cuh"

namespace satk {
namespace {

constexpr int kWarps = 4;

template <class E>
__global__ void __launch_bounds__(kWarps * 32) expanded_attend_warp_kernel(ExpandedArgs a) {
  constexpr int kQ = SATK_EXPANDED_MAX_QK / 32, kV = SATK_EXPANDED_MAX_V / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(a.T) * a.H) return;
  const int t = static_cast<int>(id / a.H), h = static_cast<int>(id % a.H);
  int64_t k0 = 0;
  int n = 0;
  if (a.R > 0 && t >= a.token_starts[0] && t < a.token_starts[a.R]) {
    int lo = 0, hi = a.R;  // the last request that starts at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.token_starts[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = min(max(a.key_starts[lo], 0), a.S), e = min(max(a.key_starts[lo + 1], b), a.S);
    k0 = b;
    n = min(max(a.row_ends[t], 0), e - b);
  }
  const int D = a.dn + a.dr;
  const E *q = static_cast<const E *>(a.q) + t * a.ld_q_t + h * a.ld_q_h;
  const E *kh = static_cast<const E *>(a.k) + h * a.ld_k_h;
  const E *vh = static_cast<const E *>(a.v) + h * a.ld_v_h;
  const E *tail = static_cast<const E *>(a.tail);
  float qv[kQ], acc[kV];
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int c = i * 32 + lane;
    qv[i] = c < D ? Elem<E>::to(q[c]) * a.scale_log2 : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) acc[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = k0; j < k0 + n; ++j) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int c = i * 32 + lane;
      if (c < D)
        s = fmaf(qv[i], Elem<E>::to(c < a.dn ? kh[j * a.ld_k_s + c] : tail[j * a.ld_tail + c - a.dn]), s);
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
    for (int i = 0; i < kV; ++i) {
      const int c = i * 32 + lane;
      if (c < a.dv) acc[i] = fmaf(p, Elem<E>::to(vh[j * a.ld_v_s + c]), acc[i]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = i * 32 + lane;
    if (c < a.dv) out[c] = Elem<E>::from(acc[i] * inv);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[id] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

int expanded_attend_warp(const ExpandedArgs &a, int dtype, cudaStream_t stream) {
  const int64_t grid = (static_cast<int64_t>(a.T) * a.H + kWarps - 1) / kWarps;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  if (dtype == SATK_BF16)
    expanded_attend_warp_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  else
    expanded_attend_warp_kernel<__half><<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a);
  return launch_status();
}

}  // namespace satk
