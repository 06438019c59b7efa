// expanded_grad.cu -- the backward pass of the expanded attention: entry points,
// the rows' statistics before it and the tail's sum over the heads after it.
#include "expanded_grad.cuh"
#include "satk_tcgen05.cuh"

namespace satk {
namespace {

constexpr int kWarps = 8;
constexpr int kRowLanes = SATK_EXPANDED_MAX_V / 8;  // lanes of a row, eight values each

// The range of row ends of one tile of tokens, ends cut to the request's keys, by a
// warp.
__device__ void tile_ends(const ExpandedGradArgs &a, int slot) {
  const int lane = threadIdx.x & 31;
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
  least = __reduce_min_sync(~0u, least);
  most = __reduce_max_sync(~0u, most);
  if (lane == 0) a.ends[slot] = make_int2(least, most);
}

// Half a warp a token and head: delta, and the normaliser in log2, head by head side
// by side (what the tiles read); the last CTAs: the tiles' row ends.  A token whose
// lse is -inf saw nothing: its row end counts as 0 wherever this is read, so a NaN of
// its own cannot get out.  VEC: rows of whole 16-byte chunks.
template <class E, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) grad_stats_kernel(ExpandedGradArgs a, unsigned row_blocks, int slots) {
  let_next_kernel_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= row_blocks) {
    const int slot = static_cast<int>(blockIdx.x - row_blocks) * kWarps + warp;
    if (slot < slots) tile_ends(a, slot);
    return;
  }
  const int64_t id = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * 2 + lane / kRowLanes;
  const int at = lane % kRowLanes;
  const unsigned lanes = ((1u << kRowLanes) - 1) << (lane - at);  // of this row
  float sum = 0.f;
  if (id < static_cast<int64_t>(a.f.T) * a.f.H) {
    const int64_t t = id / a.f.H;
    const int h = static_cast<int>(id - t * a.f.H);
    const E *dout = static_cast<const E *>(a.dout) + t * a.ld_do_t + h * a.ld_do_h;
    const E *out = static_cast<const E *>(a.f.out) + t * a.f.ld_out_t + h * a.f.ld_out_h;
    if (VEC) {
      if (at * 8 < a.f.dv) {
        Pack8<E> x, y;
        x.u = *reinterpret_cast<const uint4 *>(dout + at * 8);
        y.u = *reinterpret_cast<const uint4 *>(out + at * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 u = Elem<E>::to2(x.h[i]), v = Elem<E>::to2(y.h[i]);
          sum = fmaf(u.x, v.x, fmaf(u.y, v.y, sum));
        }
      }
    } else {
      for (int c = at; c < a.f.dv; c += kRowLanes) sum = fmaf(Elem<E>::to(dout[c]), Elem<E>::to(out[c]), sum);
    }
#pragma unroll
    for (int d = kRowLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(lanes, sum, d);
    if (at == 0)
      a.stats[static_cast<int64_t>(h) * a.f.T + t] =
          make_float2(a.f.lse[id] * kLog2e, sum - (a.dlse != nullptr ? a.dlse[id] : 0.f));
  }
}

// The heads' tails in one order, N values a thread.
template <class E, int N>
__global__ void __launch_bounds__(256) grad_tail_kernel(ExpandedGradArgs a, int64_t n) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * N;
  wait_for_previous_kernel();
  if (i >= n) return;
  float sum[N] = {};
#pragma unroll 4
  for (int h = 0; h < a.f.H; ++h) {
    const float *from = a.tails + h * n + i;
    if (N == 4) {
      const float4 x = *reinterpret_cast<const float4 *>(from);
      sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w;
    } else {
      sum[0] += *from;
    }
  }
  E *to = static_cast<E *>(a.dtail) + i / a.f.dr * a.ld_dtail + i % a.f.dr;
#pragma unroll
  for (int x = 0; x < N; ++x) to[x] = Elem<E>::from(sum[x]);
}

template <class E>
int launch_stats(const ExpandedGradArgs &a, cudaStream_t stream) {
  const int64_t rows = (static_cast<int64_t>(a.f.T) * a.f.H + 2 * kWarps - 1) / (2 * kWarps);
  const int64_t slots = tile_slots(a.f.T, a.f.R, kGradTokens), grid = rows + (slots + kWarps - 1) / kWarps;
  if (grid > INT32_MAX || slots > INT32_MAX) return SATK_EUNSUPPORTED;
  const bool vec = a.f.dv % 8 == 0 && rows_of_16_bytes(a.dout, a.f.T, a.ld_do_t, a.f.H, a.ld_do_h) &&
                   rows_of_16_bytes(a.f.out, a.f.T, a.f.ld_out_t, a.f.H, a.f.ld_out_h);
  const auto kernel = vec ? grad_stats_kernel<E, true> : grad_stats_kernel<E, false>;
  kernel<<<static_cast<unsigned>(grid), kWarps * 32, 0, stream>>>(a, static_cast<unsigned>(rows),
                                                                static_cast<int>(slots));
  return launch_status();
}

template <class E>
int launch_tail(const ExpandedGradArgs &a, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(a.f.S) * a.f.dr;
  const int each = a.f.dr % 4 == 0 ? 4 : 1;
  const int64_t grid = (n / each + 255) / 256;
  if (n == 0) return SATK_OK;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  return launch_early(each == 4 ? grad_tail_kernel<E, 4> : grad_tail_kernel<E, 1>, static_cast<unsigned>(grid),
                      256, 0, stream, a, n);
}

}  // namespace

int expanded_grad_prepare(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  return dtype == SATK_BF16 ? launch_stats<__nv_bfloat16>(a, stream) : launch_stats<__half>(a, stream);
}

int expanded_grad_tail(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  return dtype == SATK_BF16 ? launch_tail<__nv_bfloat16>(a, stream) : launch_tail<__half>(a, stream);
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
