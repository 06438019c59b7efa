// expanded_grad_tokens.cu -- gradient of the queries of the expanded attention on
// the tensor cores.
//
// A CTA takes 128 tokens of one request and head and goes over their keys in tiles
// of 128:
//   S[token, key] = Q [K | tail]^T         dP[token, key] = dO V^T
//   dS = exp2(scale S - lse) (dP - delta)  dQ += dS [K | tail]
// A token is a TMEM lane and a thread.  dS, rounded to the inputs' type, is the A
// operand of the second product from tensor memory; S 128, dP 128, dQ up to 192
// and dS 64 columns fill it.  (Wider queries have dS in the place of S.)  While dS
// of a tile is computed, the scores of the next one are.
//
// S and dP are computed again, as in the kernel of the keys: seven products where
// five would do, and no sum of dQ over CTAs, whose order would change the result.
//
// Bounded by the tensor core: 2048 cycles of products a 128 x 128 tile at 192
// query/key and 128 value columns.
#include "expanded_grad_mma.cuh"

namespace satk {
namespace {

constexpr int kPanel = kTile * 128;  // bytes of 64 columns of a tile
constexpr int kMaxBuffers = 2;

struct TokensMma {
  ExpandedGradArgs a;
  GradShape s;
  int k_buffers, v_buffers;
  int early;  // the next tile's scores before this one's dQ
  CUtensorMap q, dout, k, tail, v;
};

struct Small {
  uint64_t own, k_full[kMaxBuffers][kMaxPanels], k_empty[kMaxBuffers][kMaxPanels];
  uint64_t v_full[kMaxBuffers], v_empty[kMaxBuffers], looked[kMaxBuffers];
  uint64_t s_full, s_read, dp_full, ready, dq_done, issued;
  int low[8], high[8];
  int odd_key;   // the first key that is not finite
  int place[4];  // first key, keys, first token, tokens
  uint32_t tmem;
  int dead;
};

template <class E>
__global__ void __launch_bounds__(kGradThreads, 1)
    expanded_grad_tokens_kernel(const __grid_constant__ TokensMma m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const ExpandedGradArgs &a = m.a;
  const ExpandedArgs &f = a.f;
  const int panels = m.s.panels, v_panels = m.s.v_panels;
  const uint32_t base = smem_addr(smem);
  const int do_at = panels * kPanel, k_at = do_at + v_panels * kPanel;
  const int v_at = k_at + m.k_buffers * panels * kPanel;
  Small &sm = *reinterpret_cast<Small *>(smem + v_at + m.v_buffers * v_panels * kPanel);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % f.H;
  const int D = f.dn + f.dr;

  if (blockIdx.x >= gridDim.x - f.H) {
    rows_outside(f.token_starts, f.R, f.T, [&](int64_t t) {
      E *q = static_cast<E *>(a.dq) + t * a.ld_dq_t + h * a.ld_dq_h;
      for (int c = lane; c < D; c += 32) q[c] = Elem<E>::from(0.f);
    });
    return;
  }
  if (warp == 0) {
    const int slot = blockIdx.x / f.H;
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
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(bar(sm.own), 1);
    for (int b = 0; b < kMaxBuffers; ++b) {
      for (int p = 0; p < kMaxPanels; ++p) {
        mbar_init(bar(sm.k_full[b][p]), 1);
        mbar_init(bar(sm.k_empty[b][p]), 1);
      }
      mbar_init(bar(sm.v_full[b]), 1);
      mbar_init(bar(sm.v_empty[b]), 1);
      mbar_init(bar(sm.looked[b]), 64);
    }
    mbar_init(bar(sm.s_full), 1);
    mbar_init(bar(sm.s_read), 256);
    mbar_init(bar(sm.dp_full), 1);
    mbar_init(bar(sm.ready), 256);
    mbar_init(bar(sm.dq_done), 1);
    mbar_init(bar(sm.issued), 1);
    sm.dead = 0;
    sm.odd_key = INT32_MAX;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const int key0 = sm.place[0], keys = sm.place[1], t0 = sm.place[2], n_tokens = sm.place[3];
  if (n_tokens == 0) return;

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
  const int n = (high + kTile - 1) / kTile;
  const uint32_t dp_at = tmem + 128, dq_at = tmem + 256;
  // dS: 32 columns of each half of the keys
  const uint32_t ds_at = m.early ? dq_at + D : tmem, ds_half = m.early ? 32 : 64;

  // 168 registers a thread at launch: 256 x 208 + 128 x 88 = 384 x 168.
  if (warp < 8) regs_raise<208>(); else regs_lower<88>();
  if (warp < 8) {
    // ------------------------------------------------------------- dS, results
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 scale2 = make_float2(f.scale_log2, f.scale_log2);
    const float2 less = make_float2(-st.x, -st.x), delta = make_float2(-st.y, -st.y);
    for (int i = 0; i < n; ++i) {
      const int k0 = i * kTile + half * 64;
      uint32_t s[64];
      mbar_wait(bar(sm.s_full), i & 1, dead);
      __syncwarp();
      tc_fence_after();
      tmem_ld32(s, 0, tmem + half * 64 + lanes);
      tmem_ld32(s, 32, tmem + half * 64 + 32 + lanes);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar(sm.s_read));
#pragma unroll
      for (int x = 0; x < 32; ++x) {
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
      uint32_t packed[32];
      const bool masked = __any_sync(~0u, k0 + 64 > end);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32];
        tmem_ld32(dp, 0, dp_at + half * 64 + c * 32 + lanes);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int y = c * 32 + 2 * x;
          float2 d = __fmul2_rn(
              make_float2(__uint_as_float(s[y]), __uint_as_float(s[y + 1])),
              __fadd2_rn(make_float2(__uint_as_float(dp[2 * x]), __uint_as_float(dp[2 * x + 1])), delta));
          if (masked) {
            if (k0 + y >= end) d.x = 0.f;
            if (k0 + y + 1 >= end) d.y = 0.f;
          }
          union {
            typename Elem<E>::T2 h;
            uint32_t u;
          } pk;
          pk.h = Elem<E>::from2(d.x, d.y);
          packed[c * 16 + x] = pk.u;
        }
      }
      if (i > 0) {  // dS of the tile before has been used
        mbar_wait(bar(sm.dq_done), (i - 1) & 1, dead);
        __syncwarp();
        tc_fence_after();
      }
      tmem_st32(ds_at + half * ds_half + lanes, packed, 0);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(sm.ready));
    }
    if (n > 0) {
      mbar_wait(bar(sm.dq_done), (n - 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
    }
    const bool nan = *dead != 0 || *static_cast<volatile int *>(&sm.odd_key) < end;
    E *to = static_cast<E *>(a.dq) + static_cast<int64_t>(t) * a.ld_dq_t + h * a.ld_dq_h;
    for (int c = half * 16; c < D; c += 32) {
      uint32_t x[16];
      if (n > 0) {
        tmem_ld16(x, dq_at + c + lanes);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int y = 0; y < 16; ++y) x[y] = 0;
      }
      if (mine) store16<E>(to + c, x, nan ? NAN : a.scale, m.s.vec_q);
      __syncwarp();
    }
    tc_fence_before();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_leader()) {
      constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
      constexpr uint32_t d_s = mma_desc(bf16, false, false, kTile, kTile);
      const uint64_t q_desc = tile_desc(base, 16, 1024), o_desc = tile_desc(base + do_at, 16, 1024);
      const uint64_t k_cols = tile_desc(base + k_at, 16, 1024), v_cols = tile_desc(base + v_at, 16, 1024);
      const uint64_t k_rows = tile_desc(base + k_at, kPanel, 1024);
      const int nope_last = m.s.nope_panels - 1, cut = f.dn - nope_last * 64;
      const int v_last = f.dv - (v_panels - 1) * 64;
      auto columns = [&](int p) { return p > nope_last ? f.dr : p == nope_last ? cut : 64; };
      auto scores = [&](int i) {
        const int b = i % m.k_buffers;
        uint64_t q = q_desc, k = k_cols + (b * panels * kPanel >> 4);
        for (int p = 0; p < panels; ++p, q += kPanel >> 4, k += kPanel >> 4) {
          mbar_wait(bar(sm.k_full[b][p]), (i / m.k_buffers) & 1, dead);
          tc_fence_after();
          const int steps = columns(p) >> 4;
          for (int x = 0; x < steps; ++x) mma_ss(tmem, q + 2 * x, k + 2 * x, d_s, p > 0 || x > 0);
        }
        tc_commit(bar(sm.s_full));
      };
      auto dps = [&](int i) {
        const int b = i % m.v_buffers;
        mbar_wait(bar(sm.v_full[b]), (i / m.v_buffers) & 1, dead);
        tc_fence_after();
        product_over_columns(dp_at, o_desc, kPanel, v_cols + (b * v_panels * kPanel >> 4), kPanel, d_s,
                             v_panels, v_panels, 64, v_last);
        tc_commit(bar(sm.dp_full));
        tc_commit(bar(sm.v_empty[b]));
      };
      if (n > 0) {
        mbar_wait(bar(sm.own), 0, dead);
        scores(0);
        dps(0);
      }
      for (int i = 0; i < n; ++i) {
        if (m.early && i + 1 < n) {
          mbar_wait(bar(sm.s_read), i & 1, dead);
          tc_fence_after();
          scores(i + 1);
        }
        const int b = i % m.k_buffers;
        mbar_wait(bar(sm.looked[b]), (i / m.k_buffers) & 1, dead);
        mbar_wait(bar(sm.ready), i & 1, dead);
        tc_fence_after();
        // A panel's columns at a time, so that its place is free for the next tile's.
        uint64_t k = k_rows + (b * panels * kPanel >> 4);
        uint32_t d = dq_at;
        for (int p = 0; p < panels; ++p, k += kPanel >> 4) {
          const int cols = columns(p);
          const uint32_t desc = mma_desc(bf16, false, true, kTile, cols);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mma_ts(d, ds_at + (x >> 2) * ds_half + (x & 3) * 8, k + 128 * x, desc, i > 0 || x > 0);
          d += cols;
          tc_commit(bar(sm.k_empty[b][p]));
        }
        tc_commit(bar(sm.dq_done));
        if (i + 1 < n) {
          if (!m.early) scores(i + 1);
          dps(i + 1);
        }
      }
      tc_commit(bar(sm.issued));
      mbar_drain(bar(sm.issued), 0);
    }
    __syncwarp();
  } else if (warp == 9) {
    // -------------------------------------------------------------------- loads
    const uint32_t leader = elect_leader();
    if (n > 0) {
      if (lane == 0) mbar_expect(bar(sm.own), (panels + v_panels) * kPanel);
      __syncwarp();
      for (int p = 0; p < panels; ++p)
        tma_box3(leader, base + p * kPanel, &m.q, p < m.s.nope_panels ? p * 64 : f.dn, h, t0, bar(sm.own));
      for (int p = 0; p < v_panels; ++p)
        tma_box3(leader, base + do_at + p * kPanel, &m.dout, p * 64, h, t0, bar(sm.own));
    }
    for (int i = 0; i < n; ++i) {
      const int key = key0 + i * kTile, b = i % m.k_buffers, vb = i % m.v_buffers;
      for (int p = 0; p < panels; ++p) {
        if (i >= m.k_buffers) mbar_wait(bar(sm.k_empty[b][p]), (i / m.k_buffers - 1) & 1, dead);
        __syncwarp();
        const uint32_t full = bar(sm.k_full[b][p]), to = base + k_at + (b * panels + p) * kPanel;
        if (lane == 0) mbar_expect(full, kPanel);
        __syncwarp();
        if (p < m.s.nope_panels) tma_box3(leader, to, &m.k, p * 64, h, key, full);
        else tma_box(leader, to, &m.tail, 0, key, full);
      }
      if (i >= m.v_buffers) mbar_wait(bar(sm.v_empty[vb]), (i / m.v_buffers - 1) & 1, dead);
      __syncwarp();
      if (lane == 0) mbar_expect(bar(sm.v_full[vb]), v_panels * kPanel);
      __syncwarp();
      for (int p = 0; p < v_panels; ++p)
        tma_box3(leader, base + v_at + (vb * v_panels + p) * kPanel, &m.v, p * 64, h, key, bar(sm.v_full[vb]));
    }
    if (n > 0) mbar_drain(bar(sm.own), 0);
    for (int i = max(0, n - m.k_buffers); i < n; ++i)
      for (int p = 0; p < panels; ++p) mbar_drain(bar(sm.k_full[i % m.k_buffers][p]), (i / m.k_buffers) & 1);
    for (int i = max(0, n - m.v_buffers); i < n; ++i)
      mbar_drain(bar(sm.v_full[i % m.v_buffers]), (i / m.v_buffers) & 1);
  } else {
    // ----------------------------------------------------------------- key rows
    // Where some token does not see some key, a key that is not finite would turn a
    // 0 of dS into NaN: it is cleared, and the tokens that do see it get NaN.
    for (int i = 0; i < n; ++i) {
      const int b = i % m.k_buffers;
      for (int p = 0; p < panels; ++p) mbar_wait(bar(sm.k_full[b][p]), (i / m.k_buffers) & 1, dead);
      if (i * kTile + kTile > low) {
        unsigned char *k = smem + k_at + b * panels * kPanel;
        for (int y = (warp - 10) * 64 + lane; y < (warp - 9) * 64; y += 32)
          if (row_is_odd<E>(k, y, panels, kPanel)) {
            clear_row(k, y, panels, kPanel);
            atomicMin(&sm.odd_key, i * kTile + y);
          }
        fence_async_shared();
      }
      mbar_arrive(bar(sm.looked[b]));
    }
  }
  __syncthreads();
  if (warp == 8) tmem_free(tmem, 512);
}

bool layout(const ExpandedGradArgs &a, TokensMma &m, int &smem) {
  const int own = (m.s.panels + m.s.v_panels) * kPanel, small = static_cast<int>(sizeof(Small));
  const int k = m.s.panels * kPanel, v = m.s.v_panels * kPanel, left = kSmemLimit - own - small;
  m.k_buffers = left >= 2 * k + v ? 2 : 1;
  m.v_buffers = left >= m.k_buffers * k + 2 * v ? 2 : 1;
  m.early = m.k_buffers == 2 && 128 + 128 + a.f.dn + a.f.dr + 64 <= 512;
  smem = own + m.k_buffers * k + m.v_buffers * v + small;
  return smem <= kSmemLimit;
}

template <class E>
int launch(const TokensMma &m, int smem, cudaStream_t stream) {
  if (!allow_smem(expanded_grad_tokens_kernel<E>, smem, kSmemLimit)) return SATK_ECUDA;
  const int64_t grid = (tile_slots(m.a.f.T, m.a.f.R, kTile) + 1) * m.a.f.H;
  if (grid > INT32_MAX) return SATK_EUNSUPPORTED;
  expanded_grad_tokens_kernel<E><<<static_cast<unsigned>(grid), kGradThreads, smem, stream>>>(m);
  return launch_status();
}

}  // namespace

bool rows_of_16_bytes(const void *p, int64_t n, int64_t ld, int64_t H, int64_t ld_h) {
  return aligned16(p) && (n <= 1 || ld % 8 == 0) && (H <= 1 || ld_h % 8 == 0);
}

bool grad_map(CUtensorMap *to, bool bf16, const void *p, int cols, int64_t H, int64_t n, int64_t ld,
              int64_t ld_h, int rows) {
  // Strides of dimensions of one are free: any multiple of 16 bytes.
  return tensor_map_16bit(to, bf16, p, cols, H, H == 1 ? 1024 : ld_h, 1, n, n == 1 ? 1024 : ld, rows);
}

bool expanded_grad_tokens_fits(const ExpandedGradArgs &a, const GradShape &s) {
  TokensMma m;
  m.s = s;
  int smem;
  return layout(a, m, smem);
}

int expanded_grad_tokens(const ExpandedGradArgs &a, const GradShape &s, int dtype, cudaStream_t stream) {
  TokensMma m;
  m.a = a;
  m.s = s;
  int smem;
  const ExpandedArgs &f = a.f;
  const bool bf16 = dtype == SATK_BF16;
  if (!layout(a, m, smem)) return SATK_EUNSUPPORTED;
  if (!grad_map(&m.q, bf16, f.q, f.dn + f.dr, f.H, f.T, f.ld_q_t, f.ld_q_h, kTile) ||
      !grad_map(&m.dout, bf16, a.dout, f.dv, f.H, f.T, a.ld_do_t, a.ld_do_h, kTile) ||
      !grad_map(&m.k, bf16, f.k, f.dn, f.H, f.S, f.ld_k_s, f.ld_k_h, kTile) ||
      !grad_map(&m.v, bf16, f.v, f.dv, f.H, f.S, f.ld_v_s, f.ld_v_h, kTile) ||
      (f.dr > 0 && !tensor_map_16bit(&m.tail, bf16, f.tail, f.dr, f.S, f.S == 1 ? 1024 : f.ld_tail, kTile)))
    return SATK_ECUDA;
  return bf16 ? launch<__nv_bfloat16>(m, smem, stream) : launch<__half>(m, smem, stream);
}

}  // namespace satk
