// expanded_grad_tokens.cuh -- gradient of the queries of the expanded attention on
// the tensor cores.
//
// A CTA takes 128 tokens of one request and head and goes over their keys in tiles
// of 64:
//   S[token, key] = Q [K | tail]^T         dP[token, key] = dO V^T
//   dS = exp2(scale S - lse) (dP - delta)  dQ += dS [K | tail]
// A token is a TMEM lane and a thread.  dS, rounded to the inputs' type, replaces S
// in tensor memory and is the A operand of the second product; for requests of few
// tokens, what the rounding left is a second operand (see kFewTokens).  Q, and dO
// where there is room too, are A operands in tensor memory as well: with a tile of 64
// keys a product with both operands in shared memory takes 50 cycles a step of 16
// columns, one with A in tensor memory 36.  At 192 query/key columns: S 2 x 64, dP
// 64, Q 96, dQ 192 columns, dO in shared memory.
//
// S and dP are computed again, as in the kernel of the keys: seven products where
// five would do, and no sum of dQ over CTAs, whose order would change the result.
//
// Bounded by the tensor core: at 192 query/key and 128 value columns a 128 x 64 tile
// is 1150 cycles of products; 4096 tokens over 8192 keys, 16 heads: 1240 to 1320.  Tiles
// of 128 keys would take 2048 for twice the work, but leave room for two of them in
// shared memory, which does not hide their way there (4730 measured).
#pragma once

#include "expanded_grad_mma.cuh"

namespace satk {
namespace grad_tokens {

constexpr int kKeys = 64;  // of a tile
static_assert(kKeys == kBoxRows && kTile == 2 * kBoxRows, "boxes");
constexpr int kOwnPanel = kTile * 128, kPanel = kKeys * 128;  // bytes of 64 columns
constexpr int kMaxStages = 4;

struct Plan {
  int stages;
  int q_inside, do_inside;  // in tensor memory
};

struct Small {
  uint64_t own, full[kMaxStages], empty[kMaxStages], looked[kMaxStages];
  // (ready: a warp may be a tile ahead of another, so its arrival must not count for
  // the tile before)
  uint64_t s_full[2], dp_full, dp_read, ready[2], done, issued;
  int low[8], high[8];
  int odd_key;   // the first key that is not finite
  int place[5];  // first key, keys, first token, tokens, tokens of the request
  uint32_t tmem;
  int dead;
};

// This thread's half of a row of `cols` 16-bit columns into tensor memory.
template <class E>
__device__ __forceinline__ void row_inside(uint32_t at, const E *row, int cols, int half, bool mine) {
  for (int c = half * 16; c < cols; c += 32) {
    uint32_t x[8] = {};
    if (mine) {
      const uint4 a = *reinterpret_cast<const uint4 *>(row + c), b = *reinterpret_cast<const uint4 *>(row + c + 8);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __syncwarp();
    tmem_st8(at + c / 2, x);
  }
}

// CTA `block` of `blocks`.
template <class E>
__device__ __forceinline__ void run(const ExpandedGradArgs &a, const GradShape &shape, const Plan &m, const GradMaps &maps,
                                    unsigned char *smem, unsigned block, unsigned blocks) {
  const ExpandedArgs &f = a.f;
  const int panels = shape.panels, v_panels = shape.v_panels, stages = m.stages;
  const uint32_t base = smem_addr(smem);
  const int do_at = m.q_inside ? 0 : panels * kOwnPanel;
  const int ring_at = do_at + (m.do_inside ? 0 : v_panels * kOwnPanel);
  const int stage_bytes = (panels + v_panels) * kPanel, v_at = panels * kPanel;
  Small &sm = *reinterpret_cast<Small *>(smem + ring_at + stages * stage_bytes);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = block % f.H;
  const int D = f.dn + f.dr;

  if (block >= blocks - f.H) {
    rows_outside(f.token_starts, f.R, f.T, [&](int64_t t) {
      E *q = static_cast<E *>(a.dq) + t * a.ld_dq_t + h * a.ld_dq_h;
      for (int c = lane; c < D; c += 32) q[c] = Elem<E>::from(0.f);
    });
    return;
  }
  if (warp == 0) {
    const int slot = block / f.H;
    const int r = request_of_slot(f.token_starts, f.R, f.T, slot);
    const Span keys = span_of(f.key_starts, r, f.S), mine = span_of(f.token_starts, r, f.T);
    const int n = mine.end - mine.begin, count = (n + kTile - 1) / kTile;
    // The last tiles of a request first: they see most keys.
    const int tile = count - 1 - (slot - mine.begin / kTile - r);
    if (lane == 0) {
      const bool real = tile >= 0 && tile < count;
      sm.place[0] = keys.begin;
      sm.place[1] = keys.end - keys.begin;
      sm.place[2] = real ? mine.begin + tile * kTile : 0;
      sm.place[3] = real ? min(kTile, n - tile * kTile) : 0;
      sm.place[4] = n;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(sm.own), 1);
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar(sm.full[s]), 1);
      mbar_init(bar(sm.empty[s]), 1);
      mbar_init(bar(sm.looked[s]), 64);
    }
    mbar_init(bar(sm.s_full[0]), 1);
    mbar_init(bar(sm.s_full[1]), 1);
    mbar_init(bar(sm.dp_full), 1);
    mbar_init(bar(sm.dp_read), 256);
    mbar_init(bar(sm.ready[0]), 256);
    mbar_init(bar(sm.ready[1]), 256);
    mbar_init(bar(sm.done), 1);
    mbar_init(bar(sm.issued), 1);
    sm.dead = 0;
    sm.odd_key = INT32_MAX;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const int key0 = sm.place[0], keys = sm.place[1], t0 = sm.place[2], n_tokens = sm.place[3];
  if (n_tokens == 0) return;
  const bool few = sm.place[4] <= kFewTokens;

  // Elementwise threads: this thread's token, what it sees and its numbers.
  const int half = warp >> 2, row = threadIdx.x & 127, t = t0 + row;
  const bool mine = warp < 8 && row < n_tokens;
  float2 st = make_float2(0.f, 0.f);
  int end = 0;
  if (mine) {
    st = a.stats[static_cast<int64_t>(h) * f.T + t];
    end = st.x == -INFINITY ? 0 : min(max(f.row_ends[t], 0), keys);
    if (st.x == -INFINITY) st = make_float2(0.f, 0.f);
  }
  {
    const int lo = __reduce_min_sync(~0u, mine ? end : INT32_MAX), hi = __reduce_max_sync(~0u, end);
    if (lane == 0 && warp < 8) sm.low[warp] = lo, sm.high[warp] = hi;
  }
  if (warp == 8) tmem_alloc(smem_addr(&sm.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  int low = INT32_MAX, high = 0;
  for (int w = 0; w < 4; ++w) low = min(low, sm.low[w]), high = max(high, sm.high[w]);
  const int n = high / kKeys + (high % kKeys != 0);
  const int first_masked = low / kKeys;  // the first tile with a key that some token does not see
  const uint32_t dp_at = tmem + 2 * kKeys, dq_at = dp_at + kKeys, q_in = dq_at + D;
  const uint32_t do_in = q_in + (m.q_inside ? D / 2 : 0);
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  if (n > 0 && warp < 8) {
    if (m.q_inside)
      row_inside(q_in + lanes, static_cast<const E *>(f.q) + t * f.ld_q_t + h * f.ld_q_h, D, half, mine);
    if (m.do_inside)
      row_inside(do_in + lanes, static_cast<const E *>(a.dout) + t * a.ld_do_t + h * a.ld_do_h, f.dv, half, mine);
    tmem_wait_st();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();

  if (warp < 8) {
    // ------------------------------------------------------------- dS, results
    const float2 scale2 = make_float2(f.scale_log2, f.scale_log2);
    const float2 less = make_float2(-st.x, -st.x), delta = make_float2(-st.y, -st.y);
    for (int i = 0; i < n; ++i) {
      const int k0 = i * kKeys + half * 32, buffer = i & 1;
      const uint32_t s_at = tmem + buffer * kKeys + half * 32 + lanes;
      uint32_t s[32], dp[32], packed[16];
      mbar_wait(bar(sm.s_full[buffer]), (i >> 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
      tmem_ld32(s, 0, s_at);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
                              scale2, less);
        asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.x));  // (as grad_weight)
        asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.y));
        s[2 * x] = __float_as_uint(exp2_fast(e.x));
        s[2 * x + 1] = __float_as_uint(exp2_fast(e.y));
      }
      mbar_wait(bar(sm.dp_full), i & 1, dead);
      __syncwarp();
      tc_fence_after();
      tmem_ld32(dp, 0, dp_at + half * 32 + lanes);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(sm.dp_read));
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const float2 d = __fmul2_rn(
            make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
            __fadd2_rn(make_float2(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1])), delta));
        dp[2 * x] = __float_as_uint(d.x);
        dp[2 * x + 1] = __float_as_uint(d.y);
      }
      if (i >= first_masked) {
#pragma unroll
        for (int x = 0; x < 32; ++x)
          if (k0 + x >= end) dp[x] = 0;
      }
#pragma unroll
      for (int x = 0; x < 16; ++x)
        packed[x] = pack16<E>(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]));
      tmem_st16(s_at, packed);  // the first half of this thread's columns of S
      if (few) {  // what the rounding left: the second half
#pragma unroll
        for (int x = 0; x < 16; ++x)
          packed[x] = pack16_rest<E>(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]), packed[x]);
        tmem_st16(s_at + 16, packed);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(sm.ready[i & 1]));
    }
    if (n > 0) {
      mbar_wait(bar(sm.done), 0, dead);
      __syncwarp();
      tc_fence_after();
    }
    // A warp's rows, 64 columns a time, in turn by the two halves; the ring is free by
    // now, unless a wait was given up.
    const bool lost = n > 0 && (*dead != 0 || satk_stall_asked());
    const bool nan = *static_cast<volatile int *>(&sm.odd_key) < end;
    const int w0 = (warp & 3) * 32;
    unsigned char *turn = smem + ring_at + warp * 4096;
    E *to = static_cast<E *>(a.dq) + static_cast<int64_t>(t0 + w0) * a.ld_dq_t + h * a.ld_dq_h;
    if (lost) {
      if (half == 0) lose_rows(to, a.ld_dq_t, n_tokens - w0, D);
    } else {
      for (int c = half * 64; c < D; c += 128)
        store_rows(turn, dq_at + c + lanes, min(64, D - c), n > 0, nan ? NAN : a.scale, to + c, a.ld_dq_t,
                   n_tokens - w0, shape.vec_q != 0);
    }
    tc_fence_before();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_leader()) {
      constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
      constexpr uint32_t d_s = mma_desc(bf16, false, false, kTile, kKeys);
      const uint32_t d_q = mma_desc(bf16, false, true, kTile, shape.one_product ? D : f.dn);
      const uint32_t d_t = mma_desc(bf16, false, true, kTile, f.dr);
      const uint32_t q_low = desc_low(base, 16), o_low = desc_low(base + do_at, 16);
      const uint32_t stage_step = stage_bytes >> 4, v_step = v_at >> 4;
      const uint32_t q_steps = panel_steps(panels, shape.nope_panels, f.dn, f.dr);
      const uint32_t v_steps = panel_steps(v_panels, v_panels, f.dv, 0);
      const uint32_t tail_step = shape.nope_panels * kPanel >> 4;
      // the tiles' rows as operands over columns, and over rows (panels apart)
      const uint32_t cols_low = desc_low(base + ring_at, 16), rows_low = desc_low(base + ring_at, kPanel);
      const uint32_t full = bar(sm.full[0]), empty = bar(sm.empty[0]), looked = bar(sm.looked[0]);
      const uint32_t s_full = bar(sm.s_full[0]), dp_full = bar(sm.dp_full), dp_read = bar(sm.dp_read);
      const uint32_t ready = bar(sm.ready[0]), gap = shape.gap;
      const bool two = shape.one_product == 0, q_inside = m.q_inside != 0, do_inside = m.do_inside != 0;
      if (n > 0 && (!q_inside || !do_inside)) mbar_wait(bar(sm.own), 0, dead);
      with_shape(panels, v_panels, shape.full != 0, [&](auto np, auto vp, auto all) {
        // Tile i's place in the ring: its stage, the low words' distance, the phase.
        struct At {
          uint32_t stage = 0, low = 0, phase = 0;
        };
        auto following = [&](At x) {
          const bool wrap = x.stage + 1 == static_cast<uint32_t>(stages);
          x.stage = wrap ? 0 : x.stage + 1;
          x.low = wrap ? 0 : x.low + stage_step;
          x.phase ^= wrap ? 1 : 0;
          return x;
        };
        auto scores = [&](uint32_t buffer, At x) {
          mbar_wait(full + 8 * x.stage, x.phase, dead);
          tc_fence_after();
          const uint32_t d = tmem + buffer * kKeys, k = cols_low + x.low;
          if (q_inside)
            product_over_columns<true, np.value, all.value != 0, 0, kPanel>(d, q_in, k, d_s, q_steps, gap);
          else
            product_over_columns<false, np.value, all.value != 0, kOwnPanel, kPanel>(d, q_low, k, d_s, q_steps, gap);
          tc_commit(s_full + 8 * buffer);
        };
        auto dps = [&](At x) {
          const uint32_t v = cols_low + x.low + v_step;
          if (do_inside)
            product_over_columns<true, vp.value, all.value != 0, 0, kPanel>(dp_at, do_in, v, d_s, v_steps, 0);
          else
            product_over_columns<false, vp.value, all.value != 0, kOwnPanel, kPanel>(dp_at, o_low, v, d_s, v_steps, 0);
          tc_commit(dp_full);
        };
        auto gradients = [&](uint32_t i, At x) {
          mbar_wait(looked + 8 * x.stage, x.phase, dead);
          mbar_wait(ready + 8 * (i & 1), i >> 1 & 1, dead);
          tc_fence_after();
          const uint32_t k = rows_low + x.low;
          auto from = [&](uint32_t ds_at, bool more) {
            mma_ts_low(dq_at, ds_at, k, d_q, more);
            mma_ts_low(dq_at, ds_at + 8, k + 128, d_q, true);
            mma_ts_low(dq_at, ds_at + 32, k + 256, d_q, true);
            mma_ts_low(dq_at, ds_at + 40, k + 384, d_q, true);
            if (all.value == 0 && two) {
              const uint32_t d = dq_at + f.dn, t = k + tail_step;
              mma_ts_low(d, ds_at, t, d_t, more);
              mma_ts_low(d, ds_at + 8, t + 128, d_t, true);
              mma_ts_low(d, ds_at + 32, t + 256, d_t, true);
              mma_ts_low(d, ds_at + 40, t + 384, d_t, true);
            }
          };
          const uint32_t ds_at = tmem + (i & 1) * kKeys;
          from(ds_at, i > 0);
          if (few) from(ds_at + 16, true);
          tc_commit(empty + 8 * x.stage);
        };
        if (n == 0) return;
        At at;
        scores(0, at);
        dps(at);
        for (int i = 0; i + 1 < n; ++i) {
          const At next = following(at);
          scores(i + 1 & 1, next);
          mbar_wait(dp_read, i & 1, dead);
          tc_fence_after();
          dps(next);
          gradients(i, at);
          at = next;
        }
        gradients(n - 1, at);
      });
      tc_commit(bar(sm.done));
      tc_commit(bar(sm.issued));
      mbar_drain(bar(sm.issued), 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------------------- loads
    const uint32_t leader = elect_leader();
    const int own = ((m.q_inside ? 0 : panels) + (m.do_inside ? 0 : v_panels)) * kOwnPanel;
    if (n > 0 && own > 0) {
      if (lane == 0) mbar_expect(bar(sm.own), own);
      __syncwarp();
      for (int half = 0; half < 2; ++half) {
        const uint32_t to = base + half * (kOwnPanel / 2);
        const int token = t0 + half * kBoxRows;
        if (!m.q_inside)
          for (int p = 0; p < panels; ++p)
            tma_box3(leader, to + p * kOwnPanel, &maps.q, p < shape.nope_panels ? p * 64 : f.dn, h, token,
                     bar(sm.own));
        if (!m.do_inside)
          for (int p = 0; p < v_panels; ++p)
            tma_box3(leader, to + do_at + p * kOwnPanel, &maps.dout, p * 64, h, token, bar(sm.own));
      }
    }
    int stage = 0, around = 0;
    for (int i = 0; i < n; ++i) {
      const int key = key0 + i * kKeys;
      if (around > 0) mbar_wait(bar(sm.empty[stage]), (around - 1) & 1, dead);
      __syncwarp();
      const uint32_t full = bar(sm.full[stage]), to = base + ring_at + stage * stage_bytes;
      if (lane == 0) mbar_expect(full, stage_bytes);
      __syncwarp();
      for (int p = 0; p < shape.nope_panels; ++p) tma_box3(leader, to + p * kPanel, &maps.k, p * 64, h, key, full);
      if (f.dr > 0) tma_box(leader, to + shape.nope_panels * kPanel, &maps.tail, 0, key, full);
      for (int p = 0; p < v_panels; ++p) tma_box3(leader, to + v_at + p * kPanel, &maps.v, p * 64, h, key, full);
      if (++stage == stages) stage = 0, ++around;
    }
    if (n > 0 && own > 0) mbar_drain(bar(sm.own), 0);
    for (int i = max(0, n - stages); i < n; ++i) mbar_drain(bar(sm.full[i % stages]), (i / stages) & 1);
  } else {
    // ----------------------------------------------------------------- key rows
    // Where some token does not see some key, a key that is not finite would turn a
    // 0 of dS into NaN: it is cleared, and the tokens that do see it get NaN.
    // (Every tile is waited for and answered: a barrier waited for later than its
    // next phase but one would look like one that has not come.)
    const int y = (warp - 10) * 32 + lane;
    int stage = 0, around = 0;
    for (int i = 0; i < n; ++i) {
      mbar_wait(bar(sm.full[stage]), around & 1, dead);
      if (i >= first_masked) {
        unsigned char *k = smem + ring_at + stage * stage_bytes;
        if (row_is_odd<E>(k, y, panels, kPanel)) {
          clear_row(k, y, panels, kPanel);
          atomicMin(&sm.odd_key, i * kKeys + y);
        }
        fence_async_shared();
      }
      mbar_arrive(bar(sm.looked[stage]));
      if (++stage == stages) stage = 0, ++around;
    }
  }
  __syncthreads();
  if (warp == 8) tmem_free(tmem, 512);
}

// What fits: Q in tensor memory first, it saves most; then dO.
inline bool plan(const ExpandedGradArgs &a, const GradShape &shape, Plan &m, int &smem) {
  const int D = a.f.dn + a.f.dr, stage = (shape.panels + shape.v_panels) * kPanel;
  int columns = 3 * kKeys + D;
  m.q_inside = columns + D / 2 <= 512;
  if (m.q_inside) columns += D / 2;
  m.do_inside = columns + a.f.dv / 2 <= 512;
  const int own = ((m.q_inside ? 0 : shape.panels) + (m.do_inside ? 0 : shape.v_panels)) * kOwnPanel;
  m.stages = (kSmemLimit - own - static_cast<int>(sizeof(Small))) / stage;
  if (m.stages > kMaxStages) m.stages = kMaxStages;
  smem = own + m.stages * stage + static_cast<int>(sizeof(Small));
  return m.stages >= 2;
}

}  // namespace grad_tokens
}  // namespace satk
