// expanded_attend_mma.cu -- expanded (per-head) attention on the tensor cores.
//
// A CTA takes one head and up to 256 tokens of one request as two sub-tiles of
// 128, and goes over the keys in tiles of 128:
//   S_j[token, key] = Q_j . [K | tail]^T     j = 0, 1
//   P_j             = exp2(scale S_j - m)    m lags behind the running maximum
//   O_j            += P_j V
// While the softmax of one sub-tile runs, the products of the other one keep
// the tensor core busy.  A token is a TMEM lane and a thread, so maximum and
// sum need no exchange between threads; O is rescaled only when a score passes
// the reference by 2^8.  P_j replaces S_j in tensor memory and is the A operand
// of the second product from there; S_0, S_1, O_0, O_1 fill the 512 columns.
// Keys, tail and values come by TMA in 128-byte-swizzled panels of 64 columns x
// 128 keys, through one ring of panels in the order of their use (K of tile 0,
// V 0, K 1, V 1, ...); K panels are read K-major, V panels MN-major.
//
// Bounded by the tensor core: per 256 x 128 tile at 192 query/key and 128 value
// columns it takes 2560 cycles.  A sub-tile's own chain (scores, softmax,
// values) has to stay below that: the first half of the weights is handed over
// while the second is still computed.  4096 tokens over 8192 keys, 16 heads: 191
// us, 1.35 PFLOP/s (71 % of the measured bf16 rate); 256 CTAs of unequal length
// on 152 SMs leave 9 % idle, the rest are the CTAs' beginnings and ends.
//
// P_j is rounded to the values' type (both operands of a product have one): off by
// half a step of itself at most (bf16 2^-8, fp16 2^-11), the output by that share
// of sum p |v|, as much as its own rounding may be.  The sums take the weights
// before the rounding and stay in fp32, like the scores, the maxima and O_j.
//
// Keys past a request's end, or that only some tokens see, are masked by value.
// In tiles with such keys two warps look over the value rows first: one that is
// not finite would turn a 0 weight into NaN, so it is cleared, and the tokens
// that do see it get NaN.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax and results of the sub-tiles,
// warps 8 and 9 issue the MMAs of one sub-tile each (what one of them does
// between MMAs would otherwise leave the tensor core idle: 250 us against 186 for
// the 4096 x 8192 chunk), warp 10 the loads, warp 11 looks over value rows.
// Tiles of the last tokens, which see most keys, start first.
#include <cuda.h>
#include <type_traits>

#include "expanded_attend.cuh"
#include "satk_tcgen05.cuh"

namespace satk {
namespace {

constexpr int kRows = 128;             // tokens of a sub-tile, keys of a tile
constexpr int kPanel = kRows * 128;    // bytes of 64 columns of a tile
constexpr int kThreads = 384;
constexpr int kSmall = 2048;
constexpr int kMaxSlots = 12;
// Arrival barriers for the keys and the values of that many tiles: the ring holds
// fewer tiles (two panels each at least), so a barrier's last use is over before
// its next one.
constexpr int kTiles = 8;
constexpr float kLag = 8.f;

struct ExpandedMma {
  ExpandedArgs a;
  int nsub;          // sub-tiles: 2, or 1 where two do not fit
  int nope_panels, panels, v_panels;
  int slots;         // of the ring
  int vec;           // 16-byte aligned output rows
  CUtensorMap q, k, tail, v;
};

struct Small {
  uint64_t q_full[2], k_full[kTiles], v_full[kTiles], k_empty[kTiles], v_empty[kTiles];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], v_ready[kTiles], issued[2];
  int bad_key;           // the first key with a value row that is not finite
  int scan[12], low[8], high[8];
  int place[4];          // request's first key, its keys, first token, tokens
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(Small) <= kSmall, "small shared arrays");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Which tokens the CTA's tile has: tiles count through the requests in order.
__device__ void find_tile(const ExpandedArgs &a, int tile, int tokens, Small &sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) sm.place[3] = 0;
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
  auto tokens_of = [&](int r) {
    const int b = min(max(a.token_starts[r], 0), a.T), e = min(max(a.token_starts[r + 1], b), a.T);
    return make_int2(b, e);
  };
  int n = 0;
  for (int r = r0; r < r1; ++r) {
    const int2 t = tokens_of(r);
    n += (t.y - t.x + tokens - 1) / tokens;
  }
  int x = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sm.scan[warp] = x;
  __syncthreads();
  int before = x - n;
  for (int w = 0; w < warp; ++w) before += sm.scan[w];
  if (tile >= before && tile < before + n)
    for (int r = r0; r < r1; ++r) {
      const int2 t = tokens_of(r);
      const int count = (t.y - t.x + tokens - 1) / tokens;
      if (tile < before + count) {
        const int kb = min(max(a.key_starts[r], 0), a.S);
        const int ke = min(max(a.key_starts[r + 1], kb), a.S);
        sm.place[0] = kb;
        sm.place[1] = ke - kb;
        // the last tiles of a request first
        const int first = t.x + (count - 1 - (tile - before)) * tokens;
        sm.place[2] = first;
        sm.place[3] = min(tokens, t.y - first);
        break;
      }
      before += count;
    }
  __syncthreads();
}

// Empty rows for the tokens that no request has: the last CTAs, one a head.
template <class E>
__device__ void outside(const ExpandedArgs &a, int h) {
  const int b = a.R > 0 ? min(max(a.token_starts[0], 0), a.T) : a.T;
  // (within the tokens: the steps below past the requests' tokens stay in 32 bits)
  const int e = a.R > 0 ? min(max(a.token_starts[a.R], b), a.T) : a.T;
  for (int t = threadIdx.x >> 5; t < a.T; t += kThreads / 32) {
    if (t >= b && t < e) {
      t = ((e - 1 - t) / (kThreads / 32)) * (kThreads / 32) + t;  // the last such t below e
      continue;
    }
    const int lane = threadIdx.x & 31;
    E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h;
    for (int c = lane; c < a.dv; c += 32) out[c] = Elem<E>::from(0.f);
    if (lane == 0 && a.lse != nullptr) a.lse[static_cast<int64_t>(t) * a.H + h] = -INFINITY;
  }
}

template <class E>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_attend_mma_kernel(const __grid_constant__ ExpandedMma m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const ExpandedArgs &a = m.a;
  const uint32_t base = smem_addr(smem);
  const int q_bytes = m.panels * kPanel;
  const uint32_t ring_at = base + m.nsub * q_bytes;
  Small &sm = *reinterpret_cast<Small *>(smem + m.nsub * q_bytes + m.slots * kPanel);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.H;

  if (blockIdx.x >= gridDim.x - a.H) {
    outside<E>(a, h);
    return;
  }
  find_tile(a, blockIdx.x / a.H, m.nsub * kRows, sm);
  const int key0 = sm.place[0], keys = sm.place[1], t0 = sm.place[2], tokens = sm.place[3];
  if (tokens == 0) return;

  // Softmax threads: this thread's token and its end; tiles of each sub-tile.
  const int sub = warp >> 2, row = threadIdx.x & 127;
  const int t = t0 + sub * kRows + row;
  const bool mine = sub < m.nsub && sub * kRows + row < tokens;
  int end = mine ? min(max(a.row_ends[t], 0), keys) : INT32_MAX;
  {
    int lo = end, hi = mine ? end : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      lo = min(lo, __shfl_xor_sync(~0u, lo, d));
      hi = max(hi, __shfl_xor_sync(~0u, hi, d));
    }
    if (lane == 0 && warp < 8) sm.low[warp] = lo, sm.high[warp] = hi;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTiles; ++s) {
      mbar_init(bar(sm.k_empty[s]), m.nsub);
      mbar_init(bar(sm.v_empty[s]), m.nsub);
      mbar_init(bar(sm.k_full[s]), 1);
      mbar_init(bar(sm.v_full[s]), 1);
      mbar_init(bar(sm.v_ready[s]), 32);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(bar(sm.q_full[j]), 1);
      mbar_init(bar(sm.s_full[j]), 1);
      mbar_init(bar(sm.p_half[j]), kRows);
      mbar_init(bar(sm.p_full[j]), kRows);
      mbar_init(bar(sm.o_done[j]), 1);
    }
    mbar_init(bar(sm.issued[0]), 1);
    mbar_init(bar(sm.issued[1]), 1);
    sm.dead = 0;
    sm.bad_key = INT32_MAX;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc(smem_addr(&sm.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  int low = INT32_MAX, n_sub[2] = {0, 0};
  for (int w = 0; w < 8; ++w) {
    low = min(low, sm.low[w]);
    n_sub[w >> 2] = max(n_sub[w >> 2], (sm.high[w] + kRows - 1) / kRows);
  }
  const int n = max(n_sub[0], n_sub[1]);

  // 168 registers a thread at launch: 256 x 208 + 128 x 88 = 384 x 168.
  if (warp < 8) regs_raise<208>(); else regs_lower<88>();
  if (warp < 8) {
    // --------------------------------------------------------- softmax, results
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + sub * kRows + lanes, o_at = tmem + 256 + sub * kRows + lanes;
    const int my_tiles = sub < m.nsub ? n_sub[sub] : 0;
    // A reference beyond kFine is looked at in every tile (`move`, the maximum that
    // moves it, is then -inf), whose scores become far_exponent() / scale.
    float l = 0.f, ref = kUnset, move = kUnset;
    const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
    for (int i = 0; i < my_tiles; ++i) {
      const int k0 = i * kRows;
      uint32_t raw[kRows];
      mbar_wait(bar(sm.s_full[sub]), i & 1, dead);
      if (i > 0) mbar_wait(bar(sm.o_done[sub]), (i - 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(raw, c * 32, s_at + c * 32);
      tmem_wait_ld();
      if (__any_sync(~0u, k0 + kRows > end)) {
#pragma unroll
        for (int x = 0; x < kRows; ++x)
          if (k0 + x >= end) raw[x] = 0xff800000u;  // -inf
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < kRows; x += 2)
        m4[x >> 1 & 3] = max3(m4[x >> 1 & 3], __uint_as_float(raw[x]), __uint_as_float(raw[x + 1]));
      const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
      float less = -ref;
      if (__any_sync(~0u, mx > move)) {
        const float now = fmaxf(ref, mx);
        const float f = exp2_fast(ref - now);
        l *= f;
        ref = now;
        less = -now;
        move = now + kLag;
        if (__any_sync(~0u, fabsf(now) > kFine && now != kUnset)) {
          // Exponents over the scale: the fmaf below, which then subtracts nothing,
          // gives them back.
          const float inverse = 1.f / a.scale_log2;
#pragma unroll
          for (int x = 0; x < kRows; ++x)
            raw[x] = __float_as_uint(far_exponent(__uint_as_float(raw[x]), a.scale_log2, now) * inverse);
          less = 0.f;
          move = -INFINITY;
        }
        if (i > 0) {
          for (int c = 0; c < a.dv; c += 16) {
            uint32_t o[16];
            tmem_ld16(o, o_at + c);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
            tmem_st16(o_at + c, o);
          }
        }
      }
      const float2 less2 = make_float2(less, less);
      float2 l2[2] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const int at = c * 64 + 2 * x;
          float2 e = __ffma2_rn(make_float2(__uint_as_float(raw[at]), __uint_as_float(raw[at + 1])),
                                scale2, less2);
          e.x = exp2_fast(e.x);
          e.y = exp2_fast(e.y);
          l2[x & 1] = __fadd2_rn(l2[x & 1], e);
          union {
            typename Elem<E>::T2 h;
            uint32_t u;
          } pk;
          pk.h = Elem<E>::from2(e.x, e.y);
          p[x] = pk.u;
        }
        tmem_st32(s_at + c * 32, p, 0);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(c == 0 ? sm.p_half[sub] : sm.p_full[sub]));
      }
      l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    }
    if (sub < m.nsub) {
      if (my_tiles > 0) {
        mbar_wait(bar(sm.o_done[sub]), (my_tiles - 1) & 1, dead);
        __syncwarp();
        tc_fence_after();
      }
      if (*dead != 0) l = NAN;  // a wait was given up
      // A value row that the token sees is not finite (found before the MMAs that
      // o_done stands for): its sum of weights is as good as any.
      const bool odd = *static_cast<volatile int *>(&sm.bad_key) < end;
      const float inv = odd ? NAN : l == 0.f ? 0.f : 1.f / l;
      E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h;
      for (int c = 0; c < a.dv; c += 16) {
        uint32_t o[16];
        if (my_tiles > 0) {
          tmem_ld16(o, o_at + c);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int y = 0; y < 16; ++y) o[y] = 0;
        }
        if (mine) {
          Pack8<E> p[2];
#pragma unroll
          for (int y = 0; y < 8; ++y)
            p[y >> 2].h[y & 3] = Elem<E>::from2(__uint_as_float(o[2 * y]) * inv,
                                                __uint_as_float(o[2 * y + 1]) * inv);
          if (m.vec) {
            *reinterpret_cast<uint4 *>(out + c) = p[0].u;
            *reinterpret_cast<uint4 *>(out + c + 8) = p[1].u;
          } else {
#pragma unroll
            for (int y = 0; y < 16; ++y)
              out[c + y] = (y & 1) ? p[y >> 3].h[(y & 7) >> 1].y : p[y >> 3].h[(y & 7) >> 1].x;
          }
        }
      }
      tc_fence_before();
      if (mine && a.lse != nullptr)
        a.lse[static_cast<int64_t>(t) * a.H + h] = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
    }
  } else if (warp < 10) {
    // ---------------------------------------------------------------- MMA issue
    const int j = warp - 8;
    if (j < m.nsub && elect_leader()) {
      constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
      constexpr uint32_t ds = mma_desc(bf16, false, false, kRows, kRows);
      const uint32_t dp_full = mma_desc(bf16, false, true, kRows, 64);
      const uint32_t dp_last = mma_desc(bf16, false, true, kRows, a.dv - (m.v_panels - 1) * 64);
      const uint64_t q_desc = tile_desc(base + j * q_bytes, 16, 1024);
      const uint64_t k_desc = tile_desc(ring_at, 16, 1024), v_desc = tile_desc(ring_at, kPanel, 1024);
      const uint32_t s_col = tmem + j * kRows, o_col = tmem + 256 + j * kRows;
      const int per_tile = m.panels + m.v_panels, mine_n = n_sub[j];
      const uint32_t s_full = bar(sm.s_full[j]), o_done = bar(sm.o_done[j]);
      const uint32_t p_half = bar(sm.p_half[j]), p_full = bar(sm.p_full[j]);
      int k_slot = 0, v_slot = m.panels;  // of the next scores' and the next values' tile
      auto scores = [&]() {
        uint64_t qd = q_desc;
        int slot = k_slot;
        for (int p = 0; p < m.panels; ++p, qd += kPanel >> 4) {
          const uint64_t kd = k_desc + (slot * kPanel >> 4);
          const int cols = p < m.nope_panels ? a.dn - p * 64 : a.dr;
          if (cols >= 64) {
            mma_ss(s_col, qd, kd, ds, p > 0);
            mma_ss(s_col, qd + 2, kd + 2, ds, true);
            mma_ss(s_col, qd + 4, kd + 4, ds, true);
            mma_ss(s_col, qd + 6, kd + 6, ds, true);
          } else {
            for (int x = 0; x < cols >> 4; ++x)
              mma_ss(s_col, qd + 2 * x, kd + 2 * x, ds, p > 0 || x > 0);
          }
          if (++slot == m.slots) slot = 0;
        }
      };
      // One half of the keys of a tile: weights x values, a panel's columns at a
      // time (the ring may have the two panels apart).
      auto values = [&](int half, bool more) {
        int slot = v_slot;
        for (int p = 0; p < m.v_panels; ++p) {
          const uint64_t vd = v_desc + (slot * kPanel >> 4) + half * 512;
          const uint32_t d = o_col + p * 64, w = s_col + half * 32;
          const uint32_t dp = p == m.v_panels - 1 ? dp_last : dp_full;
          mma_ts(d, w, vd, dp, more);
          mma_ts(d, w + 8, vd + 128, dp, true);
          mma_ts(d, w + 16, vd + 256, dp, true);
          mma_ts(d, w + 24, vd + 384, dp, true);
          if (++slot == m.slots) slot = 0;
        }
      };
      if (mine_n > 0) mbar_wait(bar(sm.q_full[j]), 0, dead);
      for (int i = -1; i < n; ++i) {
        // values of tile i, scores of tile i + 1
        const int now = i & (kTiles - 1), next = (i + 1) & (kTiles - 1);
        // (A sub-tile that is done waits for the tile too before it gives it back.)
        if (i >= 0) {
          mbar_wait(bar(sm.v_ready[now]), (i / kTiles) & 1, dead);
          if (i < mine_n) {
            mbar_wait(p_half, i & 1, dead);
            tc_fence_after();
            values(0, i > 0);
            mbar_wait(p_full, i & 1, dead);
            tc_fence_after();
            values(1, true);
            tc_commit(o_done);
            tc_commit(bar(sm.v_empty[now]));
          } else {
            mbar_arrive(bar(sm.v_empty[now]));
          }
          v_slot += per_tile;
          if (v_slot >= m.slots) v_slot -= m.slots;
        }
        if (i + 1 < n) {
          mbar_wait(bar(sm.k_full[next]), ((i + 1) / kTiles) & 1, dead);
          if (i + 1 < mine_n) {
            tc_fence_after();
            scores();
            tc_commit(s_full);
            tc_commit(bar(sm.k_empty[next]));
          } else {
            mbar_arrive(bar(sm.k_empty[next]));
          }
          k_slot += per_tile;
          if (k_slot >= m.slots) k_slot -= m.slots;
        }
      }
      tc_commit(bar(sm.issued[j]));
      mbar_drain(bar(sm.issued[j]), 0);
    }
    __syncwarp();
  } else if (warp == 10) {
    // -------------------------------------------------------------------- loads
    const uint32_t leader = elect_leader();
    if (n > 0)
      for (int j = 0; j < m.nsub; ++j) {
        if (lane == 0) mbar_expect(bar(sm.q_full[j]), q_bytes);
        __syncwarp();
        for (int p = 0; p < m.panels; ++p)
          tma_box3(leader, base + j * q_bytes + p * kPanel, &m.q,
                   p < m.nope_panels ? p * 64 : a.dn, h, t0 + j * kRows, bar(sm.q_full[j]));
      }
    // The panel that had a slot before: `last` counts through them in order.
    const int per_tile = m.panels + m.v_panels;
    int slot = 0, last_tile = 0, last = -m.slots;
    for (int i = 0; i < n; ++i) {
      const int key = key0 + i * kRows;
      const uint32_t k_full = bar(sm.k_full[i % kTiles]), v_full = bar(sm.v_full[i % kTiles]);
      for (int p = 0; p < per_tile; ++p) {
        if (last == 0 || last == m.panels)
          mbar_wait(bar(last == 0 ? sm.k_empty[last_tile % kTiles] : sm.v_empty[last_tile % kTiles]),
                    (last_tile / kTiles) & 1, dead);
        if (++last == per_tile) last = 0, ++last_tile;
        __syncwarp();
        const uint32_t dst = ring_at + slot * kPanel;
        if (++slot == m.slots) slot = 0;
        if (lane == 0) {
          if (p == 0) mbar_expect(k_full, m.panels * kPanel);
          if (p == m.panels) mbar_expect(v_full, m.v_panels * kPanel);
        }
        __syncwarp();
        if (p < m.nope_panels) tma_box3(leader, dst, &m.k, p * 64, h, key, k_full);
        else if (p < m.panels) tma_box(leader, dst, &m.tail, 0, key, k_full);
        else tma_box3(leader, dst, &m.v, (p - m.panels) * 64, h, key, v_full);
      }
    }
    if (n > 0)
      for (int j = 0; j < m.nsub; ++j) mbar_drain(bar(sm.q_full[j]), 0);
    for (int i = max(0, n - kTiles); i < n; ++i) {
      mbar_drain(bar(sm.k_full[i % kTiles]), (i / kTiles) & 1);
      mbar_drain(bar(sm.v_full[i % kTiles]), (i / kTiles) & 1);
    }
  } else {
    // --------------------------------------------------------------- value rows
    int slot = 0;
    for (int i = 0; i < n; ++i) {
      slot += m.panels;
      if (slot >= m.slots) slot -= m.slots;
      const int k0 = i * kRows;
      mbar_wait(bar(sm.v_full[i % kTiles]), (i / kTiles) & 1, dead);
      for (int p = 0; p < m.v_panels; ++p) {
        unsigned char *panel = smem + (ring_at - base) + slot * kPanel;
        if (++slot == m.slots) slot = 0;
        if (k0 + kRows > low) {
          // Some token does not see some key.  A row's chunks are read from
          // another one on for every lane, clear of bank conflicts.
          for (int y = lane; y < kRows; y += 32) {
            unsigned char *v = panel + y * 128;
            typename Elem<E>::T2 sum = Elem<E>::from2(0.f, 0.f), zero = sum;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              Pack8<E> c;
              c.u = *reinterpret_cast<const uint4 *>(v + ((x ^ (y & 7)) << 4));
#pragma unroll
              for (int z = 0; z < 4; ++z) sum = __hfma2(c.h[z], zero, sum);  // NaN: not finite
            }
            const float2 f = Elem<E>::to2(sum);
            if (!(f.x == 0.f && f.y == 0.f)) {
              for (int x = 0; x < 8; ++x)
                *reinterpret_cast<uint4 *>(v + (x << 4)) = make_uint4(0, 0, 0, 0);
              atomicMin(&sm.bad_key, k0 + y);
            }
          }
          fence_async_shared();
        }
      }
      mbar_arrive(bar(sm.v_ready[i % kTiles]));
    }
  }
  __syncthreads();
  if (warp == 8) tmem_free(tmem, 512);
}

// Sub-tiles and ring that fit into shared memory.
bool layout(const ExpandedArgs &a, ExpandedMma &m, int &smem) {
  m.nope_panels = (a.dn + 63) / 64;
  m.panels = m.nope_panels + (a.dr > 0 ? 1 : 0);
  m.v_panels = (a.dv + 63) / 64;
  for (m.nsub = 2; m.nsub >= 1; --m.nsub) {
    m.slots = (kSmemLimit - kSmall) / kPanel - m.nsub * m.panels;
    if (m.slots > kMaxSlots) m.slots = kMaxSlots;
    smem = (m.nsub * m.panels + m.slots) * kPanel + kSmall;
    // the values of a tile and the keys of the next one are in use together
    if (m.slots >= m.panels + m.v_panels) return true;
  }
  return false;
}

bool rows_aligned(const void *p, int64_t n, int64_t ld, int64_t H, int64_t ld_h) {
  return aligned16(p) && (n <= 1 || ld % 8 == 0) && (H <= 1 || ld_h % 8 == 0);
}

template <class E>
int launch(const ExpandedMma &m, int smem, cudaStream_t stream) {
  const ExpandedArgs &a = m.a;
  if (!allow_smem(expanded_attend_mma_kernel<E>, smem, kSmemLimit)) return SATK_ECUDA;
  const int64_t grid = (a.T / (m.nsub * kRows) + a.R + 1ll) * a.H;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  expanded_attend_mma_kernel<E><<<static_cast<unsigned>(grid), kThreads, smem, stream>>>(m);
  return launch_status();
}

}  // namespace

bool expanded_attend_mma_fits(const ExpandedArgs &a) {
  ExpandedMma m;
  int smem;
  return a.S > 0 && a.scale_log2 > 0.f && a.dn % 16 == 0 && a.dr % 16 == 0 && a.dv % 16 == 0 &&
         a.dr <= 64 && rows_aligned(a.q, a.T, a.ld_q_t, a.H, a.ld_q_h) &&
         rows_aligned(a.k, a.S, a.ld_k_s, a.H, a.ld_k_h) &&
         rows_aligned(a.v, a.S, a.ld_v_s, a.H, a.ld_v_h) &&
         (a.dr == 0 || rows_aligned(a.tail, a.S, a.ld_tail, 1, 0)) && layout(a, m, smem);
}

int expanded_attend_mma(const ExpandedArgs &a, int dtype, cudaStream_t stream) {
  ExpandedMma m;
  int smem;
  m.a = a;
  if (!layout(a, m, smem)) return SATK_EUNSUPPORTED;
  m.vec = rows_aligned(a.out, a.T, a.ld_out_t, a.H, a.ld_out_h);
  const bool bf16 = dtype == SATK_BF16;
  // Strides of dimensions of one are free: any multiple of 16 bytes.
  auto map = [&](CUtensorMap *to, const void *p, int cols, int64_t n, int64_t ld, int64_t ld_h) {
    return tensor_map_16bit(to, bf16, p, cols, a.H, a.H == 1 ? 1024 : ld_h, 1, n, n == 1 ? 1024 : ld,
                            kRows);
  };
  if (!map(&m.q, a.q, a.dn + a.dr, a.T, a.ld_q_t, a.ld_q_h) ||
      !map(&m.k, a.k, a.dn, a.S, a.ld_k_s, a.ld_k_h) ||
      !map(&m.v, a.v, a.dv, a.S, a.ld_v_s, a.ld_v_h) ||
      (a.dr > 0 && !tensor_map_16bit(&m.tail, bf16, a.tail, a.dr, a.S, a.S == 1 ? 1024 : a.ld_tail,
                                     kRows)))
    return SATK_ECUDA;
  return bf16 ? launch<__nv_bfloat16>(m, smem, stream) : launch<__half>(m, smem, stream);
}

}  // namespace satk
