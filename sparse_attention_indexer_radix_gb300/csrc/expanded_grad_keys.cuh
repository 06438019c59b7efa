// expanded_grad_keys.cuh -- gradients of keys, tail and values of the expanded
// attention on the tensor cores.
//
// A CTA takes 128 keys of one request and head and goes over the tokens that see
// any of them in tiles of 64:
//   S[key, token]  = [K | tail] Q^T        dP[key, token] = V dO^T
//   P  = exp2(scale S - lse)               dS = P (dP - delta)
//   dV += P dO                             dK += dS Q
// The keys are the M side throughout, so P and dS need no exchange between
// threads: rounded to the inputs' type (as the forward pass rounds P: off by half
// a step of themselves), they replace S in tensor memory and are the A operand of
// the second products; for requests of few tokens, what the rounding left is a second
// operand (see kFewTokens).  dV and dK stay in tensor memory for the whole call.  S has
// two buffers where they fit (two of 64 columns, dP 64, dV 128, dK 192: 512), so
// that the scores of the next tile are computed while P and dS of this one are.
//
// The tail's gradient is summed over the heads by a kernel of its own, from a part
// of each head: no atomics, the same bits every time.
//
// Bounded by the tensor core: at 192 query/key and 128 value columns a 128 x 64 tile
// is 1580 cycles of products, of which the scores and dP, both operands in shared
// memory, take 1000 (50 a step of 16 columns: 6 KB at 128 bytes a cycle).  4096
// tokens over 8192 keys, 16 heads: 1700 cycles a tile; with the queries' CTAs 600
// us, the tensor core 67 % active.  The rest are the CTAs' beginnings (5 thousand
// cycles) and ends (5.5).
#pragma once

#include "expanded_grad_mma.cuh"

namespace satk {
namespace grad_keys {

constexpr int kTokens = kGradTokens;  // of a tile
static_assert(kTokens == kBoxRows && kTile == 2 * kBoxRows, "boxes");
static_assert(kFewTokens <= kTokens, "requests of few tokens have one tile of them");
constexpr int kKeyPanel = kTile * 128, kTokenPanel = kTokens * 128;  // bytes
constexpr int kMaxStages = 4;

struct Plan {
  int stages, score_buffers;
};

// A tile's tokens (rows of 16 bytes): -lse in log2, -delta, row ends (0 for one that sees nothing).
struct alignas(16) Tokens {
  float less[kTokens], delta[kTokens];
  int end[kTokens];
};

struct Small {
  uint64_t own, full[kMaxStages], empty[kMaxStages], tokens[kMaxStages], looked[kMaxStages];
  // (ready: a warp may be a tile ahead of another, so its arrival must not count for
  // the tile before)
  uint64_t s_full[2], dp_full, dp_read, ready[2], done, issued;
  int least[kMaxStages][2];  // smallest row end of each half of a tile
  int odd_end;               // keys below it are seen by a token that is not finite
  int place[6];              // first key (of all), first key of the request's, keys in the tile,
                             // keys of the request, first token, tokens
  int slots;                 // first tile of the request's tokens in the table of ends
  int live;                  // tiles with a token that sees the keys
  uint32_t tmem;
  int dead;
};

// The tiles of tokens that see a key of this CTA's, in order, by a whole warp.
struct LiveTiles {
  const int2 *ends;
  int count, first_key, base = -32;
  unsigned mask = 0;
  __device__ __forceinline__ int next() {
    while (mask == 0) {
      base += 32;
      if (base >= count) return -1;
      const int i = base + (threadIdx.x & 31);
      mask = __ballot_sync(~0u, i < count && ends[i].y > first_key);
    }
    const int bit = __ffs(mask) - 1;
    mask &= mask - 1;
    return base + bit;
  }
};

// P and dS of n tiles, by the elementwise warps.  A warp has 32 keys (its TMEM lanes)
// and half of each tile's tokens; a thread two of every eight tokens of four keys, so
// that it needs few tokens' numbers: a load that all lanes share costs shared memory
// as much as any other, and the products need all that it delivers (one key and 32
// tokens a thread: 451 cycles of loads a tile).
template <class E, bool FEW>
__device__ __forceinline__ void weigh(const ExpandedArgs &f, Small &sm, Tokens *tokens, uint32_t tmem, uint32_t dp_at,
                                      int key0, int n, int buffers, int stages, int half, uint32_t lanes) {
  const float2 scale2 = make_float2(f.scale_log2, f.scale_log2);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int stage = 0, around = 0;
  for (int i = 0; i < n; ++i) {
    const int buffer = buffers == 2 ? i & 1 : 0;
    const uint32_t s_at = tmem + buffer * kTokens + half * 32 + lanes;
    const Tokens &tk = tokens[stage];
    uint32_t s[32], dp[32], p16[16], d16[16];
    mbar_wait(bar(sm.tokens[stage]), around & 1, dead);
    const bool masked = sm.least[stage][half] < key0 + kTile;
    float2 less[4], delta[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      less[j] = *reinterpret_cast<const float2 *>(tk.less + half * 32 + 8 * j + 2 * (lane & 3));
      delta[j] = *reinterpret_cast<const float2 *>(tk.delta + half * 32 + 8 * j + 2 * (lane & 3));
    }
    mbar_wait(bar(sm.s_full[buffer]), (buffers == 2 ? i >> 1 : i) & 1, dead);
    __syncwarp();
    tc_fence_after();
    tmem_ld_pairs(s, 0, s_at);
    tmem_ld_pairs(s, 16, s_at + (16u << 16));
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
                            scale2, less[x >> 1 & 3]);
      asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.x));  // (as grad_weight)
      asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.y));
      s[2 * x] = __float_as_uint(exp2_fast(e.x));
      s[2 * x + 1] = __float_as_uint(exp2_fast(e.y));
    }
    mbar_wait(bar(sm.dp_full), i & 1, dead);
    __syncwarp();
    tc_fence_after();
    tmem_ld_pairs(dp, 0, dp_at + half * 32 + lanes);
    tmem_ld_pairs(dp, 16, dp_at + half * 32 + lanes + (16u << 16));
    tmem_wait_ld();
    tc_fence_before();
    mbar_arrive(bar(sm.dp_read));
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float2 d = __fmul2_rn(
          make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
          __fadd2_rn(make_float2(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1])),
                     delta[x >> 1 & 3]));
      dp[2 * x] = __float_as_uint(d.x);
      dp[2 * x + 1] = __float_as_uint(d.y);
    }
    if (masked) {
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int2 end = *reinterpret_cast<const int2 *>(tk.end + half * 32 + 8 * (x >> 1 & 3) + 2 * (lane & 3));
        const int key = key0 + (warp & 3) * 32 + (x >> 3) * 16 + (x & 1) * 8 + (lane >> 2);
        if (key >= end.x) s[2 * x] = dp[2 * x] = 0;
        if (key >= end.y) s[2 * x + 1] = dp[2 * x + 1] = 0;
      }
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      p16[x] = pack16<E>(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]));
      d16[x] = pack16<E>(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]));
    }
    // This half's 32 columns of scores become 16 of P and 16 of dS.
    tmem_st_packed(s_at, p16, 0);
    tmem_st_packed(s_at + (16u << 16), p16, 8);
    tmem_st_packed(s_at + 16, d16, 0);
    tmem_st_packed(s_at + 16 + (16u << 16), d16, 8);
    if (FEW) {  // what their rounding left: in the place of dP
      const uint32_t rest = dp_at + half * 32 + lanes;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        p16[x] = pack16_rest<E>(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]), p16[x]);
        d16[x] = pack16_rest<E>(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1]), d16[x]);
      }
      tmem_st_packed(rest, p16, 0);
      tmem_st_packed(rest + (16u << 16), p16, 8);
      tmem_st_packed(rest + 16, d16, 0);
      tmem_st_packed(rest + 16 + (16u << 16), d16, 8);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(sm.ready[i & 1]));
    if (++stage == stages) stage = 0, ++around;
  }
}

// The same of the one tile of a request of few tokens.  Not inline: in one piece with
// the other's loop it cost that (packed prompts 128 us for 123).  (The debug build is
// relocatable: there a function of its own knows nothing of the kernel's registers.)
#ifdef SATK_DEBUG
#define SATK_APART __forceinline__
#else
#define SATK_APART __noinline__
#endif
template <class E>
__device__ SATK_APART void weigh_few(const ExpandedArgs &f, Small &sm, Tokens *tokens, uint32_t tmem, uint32_t dp_at,
                                       int key0, int buffers, int stages, int half, uint32_t lanes) {
  weigh<E, true>(f, sm, tokens, tmem, dp_at, key0, 1, buffers, stages, half, lanes);
}
#undef SATK_APART

// CTA `block` of `blocks`.
template <class E>
__device__ __forceinline__ void run(const ExpandedGradArgs &a, const GradShape &shape, const Plan &m, const GradMaps &maps,
                                    unsigned char *smem, unsigned block, unsigned blocks) {
  const ExpandedArgs &f = a.f;
  const int panels = shape.panels, v_panels = shape.v_panels, stages = m.stages;
  const uint32_t base = smem_addr(smem);
  const int v_at = panels * kKeyPanel, ring_at = v_at + v_panels * kKeyPanel;
  const int stage_bytes = (panels + v_panels) * kTokenPanel, do_at = panels * kTokenPanel;
  Tokens *tokens = reinterpret_cast<Tokens *>(smem + ring_at + stages * stage_bytes);
  Small &sm = *reinterpret_cast<Small *>(tokens + stages);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = block % f.H;
  const int D = f.dn + f.dr;

  if (block >= blocks - f.H) {
    rows_outside(f.key_starts, f.R, f.S, [&](int64_t s) {
      E *k = static_cast<E *>(a.dk) + s * a.ld_dk_s + h * a.ld_dk_h;
      E *v = static_cast<E *>(a.dv) + s * a.ld_dv_s + h * a.ld_dv_h;
      float *tail = a.tails + (static_cast<int64_t>(h) * f.S + s) * f.dr;
      for (int c = lane; c < f.dn; c += 32) k[c] = Elem<E>::from(0.f);
      for (int c = lane; c < f.dv; c += 32) v[c] = Elem<E>::from(0.f);
      for (int c = lane; c < f.dr; c += 32) tail[c] = 0.f;
    });
    return;
  }
  if (warp == 0) {
    const int slot = block / f.H;
    const int r = request_of_slot(f.key_starts, f.R, f.S, slot);
    const Span keys = span_of(f.key_starts, r, f.S), mine = span_of(f.token_starts, r, f.T);
    const int64_t first = static_cast<int64_t>(slot - keys.begin / kTile - r) * kTile;
    if (lane == 0) {
      sm.place[0] = static_cast<int>(keys.begin + first);
      sm.place[1] = static_cast<int>(first);
      sm.place[2] = static_cast<int>(
          first < 0 ? 0 : max(static_cast<int64_t>(0), min(static_cast<int64_t>(kTile), keys.end - keys.begin - first)));
      sm.place[3] = keys.end - keys.begin;
      sm.place[4] = mine.begin;
      sm.place[5] = mine.end - mine.begin;
      sm.slots = mine.begin / kTokens + r;
      sm.live = 0;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(sm.own), 1);
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar(sm.full[s]), 1);
      mbar_init(bar(sm.empty[s]), 1);
      mbar_init(bar(sm.tokens[s]), 64);
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
    sm.odd_end = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const int key_at = sm.place[0], key0 = sm.place[1], rows = sm.place[2], keys = sm.place[3];
  const int token0 = sm.place[4], n_tokens = sm.place[5];
  if (rows == 0) return;
  // The keys and values are on their way while the tokens' tiles are counted.
  if (warp == 9) {
    const uint32_t leader = elect_leader();
    if (lane == 0) mbar_expect(bar(sm.own), (panels + v_panels) * kKeyPanel);
    __syncwarp();
    for (int half = 0; half < 2; ++half) {
      const uint32_t to = base + half * (kKeyPanel / 2);
      const int key = key_at + half * kBoxRows;
      for (int p = 0; p < shape.nope_panels; ++p)
        tma_box3(leader, to + p * kKeyPanel, &maps.k, p * 64, h, key, bar(sm.own));
      if (f.dr > 0) tma_box(leader, to + shape.nope_panels * kKeyPanel, &maps.tail, 0, key, bar(sm.own));
      for (int p = 0; p < v_panels; ++p)
        tma_box3(leader, to + v_at + p * kKeyPanel, &maps.v, p * 64, h, key, bar(sm.own));
    }
  }
  LiveTiles tiles{a.ends + sm.slots, (n_tokens + kTokens - 1) / kTokens, key0};
  {
    int mine = 0;
    for (int i = threadIdx.x; i < tiles.count; i += kGradThreads) mine += tiles.ends[i].y > key0;
    mine = __reduce_add_sync(~0u, mine);
    if (lane == 0 && mine > 0) atomicAdd(&sm.live, mine);
  }
  if (warp == 8) tmem_alloc(smem_addr(&sm.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const int n = sm.live, buffers = m.score_buffers;
  const bool few = n > 0 && n_tokens <= kFewTokens;
  const uint32_t dp_at = tmem + buffers * kTokens, dv_at = dp_at + kTokens;
  const uint32_t dk_at = dv_at + ((f.dv + 31) & ~31);

  if (warp < 8) {
    // ------------------------------------------------------- P and dS, results
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (few)
      weigh_few<E>(f, sm, tokens, tmem, dp_at, key0, buffers, stages, half, lanes);
    else
      weigh<E, false>(f, sm, tokens, tmem, dp_at, key0, n, buffers, stages, half, lanes);
    if (n > 0) {
      mbar_wait(bar(sm.done), 0, dead);
      __syncwarp();
      tc_fence_after();
    }
    // A warp's rows, 64 columns a time (of the tail 32), in turn by the two halves;
    // the ring is free by now, unless a wait was given up.
    const int odd = *static_cast<volatile int *>(&sm.odd_end), w0 = (warp & 3) * 32;
    const bool lost = n > 0 && (*dead != 0 || satk_stall_asked());
    const bool nan = key0 + w0 + lane < odd;
    const int64_t at = key_at + w0;
    const int mine = rows - w0;
    unsigned char *turn = smem + ring_at + warp * 4096;
    E *to_k = static_cast<E *>(a.dk) + at * a.ld_dk_s + h * a.ld_dk_h;
    E *to_v = static_cast<E *>(a.dv) + at * a.ld_dv_s + h * a.ld_dv_h;
    float *to_tail = a.tails + (static_cast<int64_t>(h) * f.S + at) * f.dr;
    if (lost) {
      lose_rows(half == 0 ? to_k : to_v, half == 0 ? a.ld_dk_s : a.ld_dv_s, mine, half == 0 ? f.dn : f.dv);
      if (half == 0) lose_rows(to_tail, f.dr, mine, f.dr);
    } else {
      int turns = 0;
      for (int c = 0; c < f.dv; c += 64)
        if ((turns++ & 1) == half)
          store_rows(turn, dv_at + c + lanes, min(64, f.dv - c), n > 0, nan ? NAN : 1.f, to_v + c, a.ld_dv_s, mine,
                     shape.vec_v != 0);
      for (int c = 0; c < f.dn; c += 64)
        if ((turns++ & 1) == half)
          store_rows(turn, dk_at + c + lanes, min(64, f.dn - c), n > 0, nan ? NAN : a.scale, to_k + c, a.ld_dk_s,
                     mine, shape.vec_k != 0);
      for (int c = 0; c < f.dr; c += 32)
        if ((turns++ & 1) == half)
          store_rows(turn, dk_at + f.dn + c + lanes, min(32, f.dr - c), n > 0, nan ? NAN : a.scale, to_tail + c,
                     f.dr, mine, true);
    }
    tc_fence_before();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_leader()) {
      constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
      constexpr uint32_t d_s = mma_desc(bf16, false, false, kTile, kTokens);
      const uint32_t d_v = mma_desc(bf16, false, true, kTile, f.dv);
      const uint32_t d_k = mma_desc(bf16, false, true, kTile, shape.one_product ? D : f.dn);
      const uint32_t d_t = mma_desc(bf16, false, true, kTile, f.dr);
      const uint32_t k_low = desc_low(base, 16), v_low = desc_low(base + v_at, 16);
      const uint32_t stage_step = stage_bytes >> 4, do_step = do_at >> 4;
      const uint32_t q_steps = panel_steps(panels, shape.nope_panels, f.dn, f.dr);
      const uint32_t v_steps = panel_steps(v_panels, v_panels, f.dv, 0);
      const uint32_t tail_step = shape.nope_panels * kTokenPanel >> 4;
      // the tiles' rows as operands over columns, and over rows (panels apart)
      const uint32_t cols_low = desc_low(base + ring_at, 16), rows_low = desc_low(base + ring_at, kTokenPanel);
      const uint32_t full = bar(sm.full[0]), empty = bar(sm.empty[0]), looked = bar(sm.looked[0]);
      const uint32_t s_full = bar(sm.s_full[0]), dp_full = bar(sm.dp_full), dp_read = bar(sm.dp_read);
      const uint32_t ready = bar(sm.ready[0]), gap = shape.gap;
      const bool two = shape.one_product == 0;
      if (n > 0) mbar_wait(bar(sm.own), 0, dead);
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
          product_over_columns<false, np.value, all.value != 0, kKeyPanel, kTokenPanel>(
              tmem + buffer * kTokens, k_low, cols_low + x.low, d_s, q_steps, gap);
          tc_commit(s_full + 8 * buffer);
        };
        auto dps = [&](At x) {
          product_over_columns<false, vp.value, all.value != 0, kKeyPanel, kTokenPanel>(
              dp_at, v_low, cols_low + x.low + do_step, d_s, v_steps, 0);
          tc_commit(dp_full);
        };
        // dV and dK of tile i from the buffer that holds its P and dS
        auto gradients = [&](uint32_t i, uint32_t buffer, At x) {
          mbar_wait(looked + 8 * x.stage, x.phase, dead);
          mbar_wait(ready + 8 * (i & 1), i >> 1 & 1, dead);
          tc_fence_after();
          const uint32_t q = rows_low + x.low, o = q + do_step;
          auto from = [&](uint32_t p_at, bool more) {
            mma_ts_low(dv_at, p_at, o, d_v, more);
            mma_ts_low(dv_at, p_at + 8, o + 128, d_v, true);
            mma_ts_low(dv_at, p_at + 32, o + 256, d_v, true);
            mma_ts_low(dv_at, p_at + 40, o + 384, d_v, true);
            mma_ts_low(dk_at, p_at + 16, q, d_k, more);
            mma_ts_low(dk_at, p_at + 24, q + 128, d_k, true);
            mma_ts_low(dk_at, p_at + 48, q + 256, d_k, true);
            mma_ts_low(dk_at, p_at + 56, q + 384, d_k, true);
            if (all.value == 0 && two) {
              const uint32_t d = dk_at + f.dn, t = q + tail_step;
              mma_ts_low(d, p_at + 16, t, d_t, more);
              mma_ts_low(d, p_at + 24, t + 128, d_t, true);
              mma_ts_low(d, p_at + 48, t + 256, d_t, true);
              mma_ts_low(d, p_at + 56, t + 384, d_t, true);
            }
          };
          from(tmem + buffer * kTokens, i > 0);
          tc_commit(empty + 8 * x.stage);
        };
        if (n == 0) return;
        At at;
        scores(0, at);
        dps(at);
        if (buffers == 2) {
          for (int i = 0; i + 1 < n; ++i) {
            const At next = following(at);
            scores(i + 1 & 1, next);
            mbar_wait(dp_read, i & 1, dead);
            tc_fence_after();
            dps(next);
            gradients(i, i & 1, at);
            at = next;
          }
          gradients(n - 1, n - 1 & 1, at);
        } else {
          for (int i = 0; i + 1 < n; ++i) {
            gradients(i, 0, at);
            at = following(at);
            scores(0, at);
            dps(at);
          }
          gradients(n - 1, 0, at);
        }
      });
      if (few) {  // one tile, in the ring's first stage: what the roundings left
        const uint32_t q = rows_low, o = q + do_step, d = dk_at + f.dn, t = q + tail_step;
#pragma unroll
        for (uint32_t x = 0; x < 4; ++x) {
          const uint32_t p_at = dp_at + (x >> 1) * 32 + (x & 1) * 8;
          mma_ts_low(dv_at, p_at, o + 128 * x, d_v, true);
          mma_ts_low(dk_at, p_at + 16, q + 128 * x, d_k, true);
          mma_ts_low_if(two, d, p_at + 16, t + 128 * x, d_t);
        }
      }
      tc_commit(bar(sm.done));
      tc_commit(bar(sm.issued));
      mbar_drain(bar(sm.issued), 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------------------- loads
    const uint32_t leader = elect_leader();
    int stage = 0, around = 0;
    for (int i = 0; i < n; ++i) {
      const int t = token0 + tiles.next() * kTokens;
      if (around > 0) mbar_wait(bar(sm.empty[stage]), (around - 1) & 1, dead);
      __syncwarp();
      const uint32_t full = bar(sm.full[stage]), to = base + ring_at + stage * stage_bytes;
      if (lane == 0) mbar_expect(full, stage_bytes);
      __syncwarp();
      for (int p = 0; p < panels; ++p)
        tma_box3(leader, to + p * kTokenPanel, &maps.q, p < shape.nope_panels ? p * 64 : f.dn, h, t, full);
      for (int p = 0; p < v_panels; ++p)
        tma_box3(leader, to + do_at + p * kTokenPanel, &maps.dout, p * 64, h, t, full);
      if (++stage == stages) stage = 0, ++around;
    }
    mbar_drain(bar(sm.own), 0);
    for (int i = max(0, n - stages); i < n; ++i)
      mbar_drain(bar(sm.full[i % stages]), (i / stages) & 1);
  } else {
    // ------------------------------------------------ the tokens' numbers and rows
    // A lane has one token of each tile.  Where some token does not see some key, a
    // row that is not finite would turn a 0 of P or dS into NaN: it is cleared, and
    // the keys that do see it get NaN.
    const int half = warp - 10, y = half * 32 + lane;
    const float2 *stats = a.stats + static_cast<int64_t>(h) * f.T;
    struct Numbers {
      float2 st;
      int end;
    };
    auto look_up = [&](int tile) {
      Numbers x{make_float2(0.f, 0.f), 0};
      const int64_t i = static_cast<int64_t>(tile) * kTokens + y;
      if (tile >= 0 && i < n_tokens) {
        x.st = stats[token0 + i];
        x.end = min(max(f.row_ends[token0 + i], 0), keys);
        if (x.st.x == -INFINITY) x = Numbers{make_float2(0.f, 0.f), 0};
      }
      return x;
    };
    Numbers now = look_up(n > 0 ? tiles.next() : -1);
    int stage = 0, around = 0;
    for (int i = 0; i < n; ++i) {
      if (around > 0) mbar_wait(bar(sm.empty[stage]), (around - 1) & 1, dead);
      tokens[stage].less[y] = -now.st.x;
      tokens[stage].delta[y] = -now.st.y;
      tokens[stage].end[y] = now.end;
      const int least = __reduce_min_sync(~0u, now.end);
      if (lane == 0) sm.least[stage][half] = least;
      __syncwarp();
      mbar_arrive(bar(sm.tokens[stage]));
      const int end = now.end;
      now = look_up(i + 1 < n ? tiles.next() : -1);
      mbar_wait(bar(sm.full[stage]), around & 1, dead);
      if (least < key0 + kTile) {
        unsigned char *q = smem + ring_at + stage * stage_bytes;
        if (row_is_odd<E>(q, y, panels + v_panels, kTokenPanel)) {
          clear_row(q, y, panels + v_panels, kTokenPanel);
          atomicMax(&sm.odd_end, end);
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

// Stages and buffers that fit; shared memory in `smem`.
inline bool plan(const ExpandedGradArgs &a, const GradShape &shape, Plan &m, int &smem) {
  const int D = a.f.dn + a.f.dr, stage = (shape.panels + shape.v_panels) * kTokenPanel;
  const int own = (shape.panels + shape.v_panels) * kKeyPanel, numbers = static_cast<int>(sizeof(Tokens));
  m.stages = (kSmemLimit - own - static_cast<int>(sizeof(Small))) / (stage + numbers);
  if (m.stages > kMaxStages) m.stages = kMaxStages;
  smem = own + m.stages * (stage + numbers) + static_cast<int>(sizeof(Small));
  m.score_buffers = 3 * kTokens + ((a.f.dv + 31) & ~31) + D <= 512 ? 2 : 1;
  return m.stages >= 2;
}

}  // namespace grad_keys
}  // namespace satk
