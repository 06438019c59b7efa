// expanded_grad_warp.cu -- the backward pass of the expanded attention, one warp
// per (key, head) for dk, dv and the head's tail, and one per (token, head) for
// dq: each goes over its request's tokens (or keys) once, its own rows and sums in
// registers, one element of every 32 per lane, all in fp32.  Any width, stride and
// alignment; rows are read again by every warp, so it is L2- and
// instruction-bound.
#include "expanded_grad.cuh"

namespace satk {
namespace {

constexpr int kWarps = 4;
constexpr int kQ = SATK_EXPANDED_MAX_QK / 32, kV = SATK_EXPANDED_MAX_V / 32;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// Element i * 32 + lane of a row of n, 0 behind it.
template <class E, int N>
__device__ __forceinline__ void load_row(float (&x)[N], const E *row, int n, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = i * 32 + lane;
    x[i] = c < n ? Elem<E>::to(row[c]) : 0.f;
  }
}
template <class E>
__device__ __forceinline__ void load_key(float (&x)[kQ], const ExpandedArgs &f, int64_t j, int h, int lane) {
  const E *k = static_cast<const E *>(f.k) + j * f.ld_k_s + h * f.ld_k_h;
  const E *tail = static_cast<const E *>(f.tail) + j * f.ld_tail;
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int c = i * 32 + lane;
    x[i] = c < f.dn ? Elem<E>::to(k[c]) : c < f.dn + f.dr ? Elem<E>::to(tail[c - f.dn]) : 0.f;
  }
}

template <class E>
__global__ void __launch_bounds__(kWarps * 32) grad_keys_warp_kernel(ExpandedGradArgs a) {
  const ExpandedArgs &f = a.f;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(f.S) * f.H) return;
  const int s = static_cast<int>(id / f.H), h = static_cast<int>(id % f.H);
  const int D = f.dn + f.dr;
  float dk[kQ] = {}, dv[kV] = {};
  const int r = request_of(f.key_starts, f.R, f.S, s);
  if (r >= 0) {
    float key[kQ], value[kV];
    load_key<E>(key, f, s, h, lane);
    load_row(value, static_cast<const E *>(f.v) + s * f.ld_v_s + h * f.ld_v_h, f.dv, lane);
    const int j = s - span_of(f.key_starts, r, f.S).begin;
    const Span tokens = span_of(f.token_starts, r, f.T);
    for (int64_t t = tokens.begin; t < tokens.end; ++t) {
      if (j >= f.row_ends[t]) continue;
      const float2 st = a.stats[static_cast<int64_t>(h) * f.T + t];
      if (st.x == -INFINITY) continue;
      float q[kQ], dout[kV], x = 0.f, dp = 0.f;
      load_row(q, static_cast<const E *>(f.q) + t * f.ld_q_t + h * f.ld_q_h, D, lane);
      load_row(dout, static_cast<const E *>(a.dout) + t * a.ld_do_t + h * a.ld_do_h, f.dv, lane);
#pragma unroll
      for (int i = 0; i < kQ; ++i) x = fmaf(q[i], key[i], x);
#pragma unroll
      for (int i = 0; i < kV; ++i) dp = fmaf(dout[i], value[i], dp);
      const float p = grad_weight(warp_sum(x), f.scale_log2, st.x);
      const float ds = p * (warp_sum(dp) - st.y);
#pragma unroll
      for (int i = 0; i < kQ; ++i) dk[i] = fmaf(ds, q[i], dk[i]);
#pragma unroll
      for (int i = 0; i < kV; ++i) dv[i] = fmaf(p, dout[i], dv[i]);
    }
  }
  E *to_k = static_cast<E *>(a.dk) + s * a.ld_dk_s + h * a.ld_dk_h;
  E *to_v = static_cast<E *>(a.dv) + s * a.ld_dv_s + h * a.ld_dv_h;
  float *to_tail = a.tails + (static_cast<int64_t>(h) * f.S + s) * f.dr;
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int c = i * 32 + lane;
    if (c < f.dn) to_k[c] = Elem<E>::from(dk[i] * a.scale);
    else if (c < D) to_tail[c - f.dn] = dk[i] * a.scale;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int c = i * 32 + lane;
    if (c < f.dv) to_v[c] = Elem<E>::from(dv[i]);
  }
}

template <class E>
__global__ void __launch_bounds__(kWarps * 32) grad_tokens_warp_kernel(ExpandedGradArgs a) {
  const ExpandedArgs &f = a.f;
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (id >= static_cast<int64_t>(f.T) * f.H) return;
  const int t = static_cast<int>(id / f.H), h = static_cast<int>(id % f.H);
  const int D = f.dn + f.dr;
  float dq[kQ] = {};
  const int r = request_of(f.token_starts, f.R, f.T, t);
  const float2 st = a.stats[static_cast<int64_t>(h) * f.T + t];
  if (r >= 0 && st.x != -INFINITY) {
    float q[kQ], dout[kV];
    load_row(q, static_cast<const E *>(f.q) + t * f.ld_q_t + h * f.ld_q_h, D, lane);
    load_row(dout, static_cast<const E *>(a.dout) + t * a.ld_do_t + h * a.ld_do_h, f.dv, lane);
    const Span keys = span_of(f.key_starts, r, f.S);
    const int64_t end = keys.begin + min(max(f.row_ends[t], 0), keys.end - keys.begin);
    for (int64_t s = keys.begin; s < end; ++s) {
      float key[kQ], value[kV], x = 0.f, dp = 0.f;
      load_key<E>(key, f, s, h, lane);
      load_row(value, static_cast<const E *>(f.v) + s * f.ld_v_s + h * f.ld_v_h, f.dv, lane);
#pragma unroll
      for (int i = 0; i < kQ; ++i) x = fmaf(q[i], key[i], x);
#pragma unroll
      for (int i = 0; i < kV; ++i) dp = fmaf(dout[i], value[i], dp);
      const float ds = grad_weight(warp_sum(x), f.scale_log2, st.x) * (warp_sum(dp) - st.y);
#pragma unroll
      for (int i = 0; i < kQ; ++i) dq[i] = fmaf(ds, key[i], dq[i]);
    }
  }
  E *to = static_cast<E *>(a.dq) + t * a.ld_dq_t + h * a.ld_dq_h;
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int c = i * 32 + lane;
    if (c < D) to[c] = Elem<E>::from(dq[i] * a.scale);
  }
}

template <class E>
int launch(const ExpandedGradArgs &a, cudaStream_t stream) {
  const int64_t keys = (static_cast<int64_t>(a.f.S) * a.f.H + kWarps - 1) / kWarps;
  const int64_t tokens = (static_cast<int64_t>(a.f.T) * a.f.H + kWarps - 1) / kWarps;
  if (keys > INT32_MAX || tokens > INT32_MAX) return SATK_EUNSUPPORTED;
  if (keys > 0) grad_keys_warp_kernel<E><<<static_cast<unsigned>(keys), kWarps * 32, 0, stream>>>(a);
  if (tokens > 0) grad_tokens_warp_kernel<E><<<static_cast<unsigned>(tokens), kWarps * 32, 0, stream>>>(a);
  return launch_status();
}

}  // namespace

int expanded_grad_warp(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  return dtype == SATK_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<__half>(a, stream);
}

}  // namespace satk
