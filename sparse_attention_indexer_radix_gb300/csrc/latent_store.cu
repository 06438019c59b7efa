// latent_store.cu -- satk_latent_store: norm of the latent, rotation of the
// tail and the scatter of both into the cache rows of a step's new tokens.
//
// One warp per token: the row's squares are summed by a warp reduction over
// values that stay in registers, so the latent is read once and the row
// written once.  16384 rows of 544 columns take 12.4 us, 3.1 TB/s of the bytes in
// and out, bound by the chain load, sum, store of each warp (two tokens a warp,
// all loads first: 13.4 us, four: 16.3); a decode step's 32 rows 2.8 us.
// The 16-byte path runs when every row starts on a 16-byte boundary and dl is
// a multiple of 8; other layouts take the same kernel with one element per
// access.
#include "latent_common.cuh"

namespace satk {
namespace {

constexpr int kStoreWarps = 8;

struct StoreArgs {
  const void *latent, *tail;
  int64_t ld_latent, ld_tail;
  int T, dl, dr;
  const float *weight;
  float eps;
  const float *cos_sin;
  int64_t n_positions;
  const int32_t *positions;
  int interleaved;
  const int32_t *slots;
  void *cache;
  int64_t cache_rows, ld_cache;
  int32_t *status;
};

template <class E, int VEC>
__global__ void __launch_bounds__(kStoreWarps * 32) latent_store_kernel(StoreArgs a) {
  constexpr int kPer = SATK_LATENT_MAX / 32;  // latent values per lane
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kStoreWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  // The row is asked for together with its slot and position.
  const int slot = a.slots[t];
  const int pos = a.cos_sin != nullptr ? a.positions[t] : 0;
  const E *x = static_cast<const E *>(a.latent) + t * a.ld_latent;
  const int half = a.dr / 2;  // the tail: lane i holds pair i (dr / 2 <= 32 pairs)
  const int i0 = a.interleaved ? 2 * lane : lane, i1 = a.interleaved ? i0 + 1 : lane + half;
  float y0 = 0.f, y1 = 0.f;
  if (lane < half) {
    const E *y = static_cast<const E *>(a.tail) + t * a.ld_tail;
    y0 = Elem<E>::to(y[i0]);
    y1 = Elem<E>::to(y[i1]);
  }
  float v[kPer];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer / VEC; ++i) {
    const int c = (i * 32 + lane) * VEC;
    if constexpr (VEC == 8) {
      Pack8<E> p;
      p.u = make_uint4(0, 0, 0, 0);
      if (c < a.dl) p.u = __ldg(reinterpret_cast<const uint4 *>(x + c));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = Elem<E>::to2(p.h[j]);
        v[i * 8 + 2 * j] = f.x;
        v[i * 8 + 2 * j + 1] = f.y;
      }
    } else {
      v[i] = c < a.dl ? Elem<E>::to(x[c]) : 0.f;
    }
  }
  if (slot < 0) return;
  const bool row_ok = slot < a.cache_rows;
  const bool pos_ok = a.cos_sin == nullptr || (pos >= 0 && pos < a.n_positions);
  if (!row_ok || !pos_ok) {
    if (lane == 0 && a.status != nullptr)
      atomicOr(a.status, row_ok ? SATK_STATUS_BAD_POSITION : SATK_STATUS_BAD_ROW);
    return;
  }
  E *out = static_cast<E *>(a.cache) + slot * a.ld_cache;
  float co = 0.f, si = 0.f;
  if (a.cos_sin != nullptr && lane < half) {
    const float *cs = a.cos_sin + static_cast<int64_t>(pos) * a.dr;
    co = __ldg(cs + lane);
    si = __ldg(cs + half + lane);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum = fmaf(v[i], v[i], sum);
  if (a.weight != nullptr) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
    const float s = rsqrtf(sum / a.dl + a.eps);
#pragma unroll
    for (int i = 0; i < kPer / VEC; ++i) {
      const int c = (i * 32 + lane) * VEC;
      if (c < a.dl) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i * VEC + j] *= s * __ldg(a.weight + c + j);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer / VEC; ++i) {
    const int c = (i * 32 + lane) * VEC;
    if (c < a.dl) {
      if constexpr (VEC == 8) {
        Pack8<E> p;
#pragma unroll
        for (int j = 0; j < 4; ++j) p.h[j] = Elem<E>::from2(v[i * 8 + 2 * j], v[i * 8 + 2 * j + 1]);
        *reinterpret_cast<uint4 *>(out + c) = p.u;
      } else {
        out[c] = Elem<E>::from(v[i]);
      }
    }
  }
  if (lane < half) {
    if (a.cos_sin != nullptr) {
      const float r0 = y0 * co - y1 * si, r1 = y0 * si + y1 * co;
      y0 = r0;
      y1 = r1;
    }
    out[a.dl + i0] = Elem<E>::from(y0);
    out[a.dl + i1] = Elem<E>::from(y1);
  }
}

}  // namespace
}  // namespace satk

extern "C" int satk_latent_store(const void *latent, int64_t ld_latent, const void *tail,
                                 int64_t ld_tail, int dtype, int64_t T, int32_t dl, int32_t dr,
                                 const float *weight, float eps, const float *cos_sin,
                                 int64_t n_positions, const int32_t *positions,
                                 int32_t interleaved, const int32_t *slots, void *cache,
                                 int64_t cache_rows, int64_t ld_cache, int32_t *status,
                                 satk_stream_t stream) {
  using namespace satk;
  if (latent == nullptr || slots == nullptr || cache == nullptr || (tail == nullptr && dr > 0) ||
      (cos_sin != nullptr && positions == nullptr) || !is_16bit(dtype) || T < 0 ||
      T > INT32_MAX || cache_rows < 0 || n_positions < 0 || dl < 1 || dr < 0 || dr % 2 != 0 ||
      (T > 1 && (ld_latent < dl || ld_tail < dr)) ||
      ld_cache < static_cast<int64_t>(dl) + dr)
    return SATK_EINVAL;
  if (dl > SATK_LATENT_MAX || dr > SATK_LATENT_TAIL_MAX) return SATK_EUNSUPPORTED;
  if (T == 0) return SATK_OK;
  StoreArgs a{latent,  tail,        ld_latent, ld_tail,     static_cast<int>(T), dl,
              dr,      weight,      eps,       dr > 0 ? cos_sin : nullptr, n_positions, positions,
              interleaved, slots,   cache,     cache_rows,  ld_cache,  status};
  const bool vec = aligned16(latent) && aligned16(cache) && dl % 8 == 0 && ld_cache % 8 == 0 &&
                   (T == 1 || ld_latent % 8 == 0);
  const unsigned grid = static_cast<unsigned>((T + kStoreWarps - 1) / kStoreWarps);
  auto launch = [&](auto kernel) {
    kernel<<<grid, kStoreWarps * 32, 0, as_stream(stream)>>>(a);
  };
  if (dtype == SATK_BF16)
    vec ? launch(latent_store_kernel<__nv_bfloat16, 8>) : launch(latent_store_kernel<__nv_bfloat16, 1>);
  else
    vec ? launch(latent_store_kernel<__half, 8>) : launch(latent_store_kernel<__half, 1>);
  return launch_status();
}
