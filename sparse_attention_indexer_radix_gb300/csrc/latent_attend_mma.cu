// latent_attend_mma.cu -- attention over latent cache rows on the tensor cores.
//
// Per group of up to 64 score columns n (heads of one token, or of several
// tokens of one request) and per tile of 64 keys:
//   S^T[key, n]  = K[key, :] . Q[n, :]            M = 64 keys,  N columns
//   P^T[key, n]  = exp2(scale S - m_n)
//   O^T[c, n]   += sum_key K[key, c] P^T[key, n]  M = 128 of the dl columns
// The keys are the M side because a token has few heads and its value rows are
// long: with heads on the M side O would be 128 lanes x dl columns, which at
// dl = 512 is all of tensor memory, and 16 heads would pay for 128.  Here O
// takes ceil(dl / 128) N columns (256 at most), S two buffers of N.  One tile
// in shared memory serves both products: K-major for S, MN-major for O.
//
// m_n is a reference that follows the running maximum lazily: it moves, and O
// and l are rescaled, only when a score passes it by more than 2^8 (a vote of
// the CTA), so most tiles need no cross-key reduction at all; l is summed per
// thread and joined once at the end.
//
// Key rows reach shared memory in two ways, each its own instantiation:
//  - BOX, where pages give runs of 8 or more keys that lie together: TMA boxes
//    of a run x 64 columns.  256 threads: warps 0-3 softmax and results, warp 4
//    issues the MMAs, warps 5-6 the boxes (every second panel of 64 columns
//    each), warp 7 brings the queries.
//  - else (selected rows, tiny pages): 16-byte asynchronous copies by eight
//    warps, each stage owned by its own warps so that several tiles are in
//    flight.  512 threads: warps 0-3 and 4 as above, 5-7 queries, 8-15 keys.
//    (TMA's gather of four rows a request moved 512 bytes in 56 cycles, a third
//    of what HBM gives an SM; the copies move twice that.)
// A row that is skipped or not in the cache is masked; if what was read in its
// place is not finite, the softmax role clears it in the tile.
//
// Split: the tiles of all groups form one line that is cut into equal pieces,
// one per SM (plan kernel); a group cut across SMs leaves unnormalised partial
// results in the workspace that a last kernel joins in a fixed order.
#include <cuda.h>
#include <type_traits>

#include "latent_attend.cuh"
#include "satk_tcgen05.cuh"

namespace satk {
namespace {

constexpr int kTile = 64;                // keys per tile
constexpr int kPanel = kTile * 128;      // bytes of 64 columns of a tile
constexpr int threads_of(bool box) { return box ? 256 : 512; }
constexpr int query_threads(bool box) { return box ? 32 : 96; }
constexpr int kSoftmax = 128;            // threads of the softmax role
constexpr int kMaxStages = 4;
constexpr int kSmall = 3072;             // barriers and per-column arrays
constexpr int kMaxTokens = 16384;        // tokens per launch (the plan's size)
constexpr int kCombineY = 16;
constexpr int kMinTiles = 2;             // tiles per SM below which no group is cut
constexpr float kUnset = -1e30f;         // reference of a column without a score
constexpr float kLag = 8.f;              // log2 by which scores may pass m_n

// One group: its tokens, the keys any of them may see, and where its tiles
// (nh head chunks after each other) start on the line.
struct Group {
  int64_t start;
  int t0, ntok, extent, req;
};

struct Plan {
  int64_t tiles, per;  // on the line, per CTA
  int ngroups, pad;
};

struct MmaArgs {
  LatentArgs a;
  Plan *plan;
  Group *group;
  float *parts;
  int nh, hc;    // head chunks and heads per chunk
  int tpg;       // tokens per group
  int np, nst;   // 64-column panels of a key row, stages
  int nb;        // 128-column blocks of a value
  int64_t part_stride;
  int q_vec, out_vec;
  int run;           // rows of a box: consecutive keys that share a block (1: copies)
  CUtensorMap rows;  // the cache, in boxes of 64 columns x run rows
};

__device__ __forceinline__ int group_tiles(const Group &g) {
  return g.extent > 0 ? (g.extent + kTile - 1) / kTile : 1;
}

__device__ __forceinline__ int64_t per_cta(int64_t tiles, int ctas) {
  const int64_t per = (tiles + ctas - 1) / ctas;
  return per < kMinTiles ? kMinTiles : per;
}

// Groups in token order, and the prefix sum of their tiles.  One CTA.
__global__ void __launch_bounds__(1024) latent_plan_kernel(MmaArgs m, int ctas) {
  const LatentArgs &a = m.a;
  __shared__ int64_t wt[32];
  __shared__ int wg[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.T + 1023) / 1024;
  const int b = min(tid * per, a.T), e = min(b + per, a.T);
  auto leader = [&](int t) {
    return m.tpg == 1 || t % m.tpg == 0 || a.req_id[t] != a.req_id[t - 1];
  };
  auto group = [&](int t) {
    Group g;
    g.t0 = t;
    g.req = a.rows == nullptr ? a.req_id[t] : 0;
    g.ntok = 0;
    g.extent = 0;
    do {
      const int end = token_end(a, t + g.ntok);
      g.extent = max(g.extent, token_extent(a, t + g.ntok, end));
      ++g.ntok;
    } while (t + g.ntok < a.T && !leader(t + g.ntok));
    return g;
  };
  Group g = {};
  int64_t tiles = 0;
  int groups = 0;
  for (int t = b; t < e; ++t)
    if (leader(t)) {
      g = group(t);
      tiles += static_cast<int64_t>(group_tiles(g)) * m.nh;
      ++groups;
    }
  int64_t st = tiles;
  int sg = groups;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, st, d);
    const int y = __shfl_up_sync(~0u, sg, d);
    if (lane >= d) st += x, sg += y;
  }
  if (lane == 31) wt[warp] = st, wg[warp] = sg;
  __syncthreads();
  int64_t all = 0;
  int n = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) st += wt[w], sg += wg[w];
    all += wt[w];
    n += wg[w];
  }
  st -= tiles;
  sg -= groups;
  Group *out = m.group;
  for (int t = b; t < e; ++t)
    if (leader(t)) {
      if (groups > 1) g = group(t);
      g.start = st;
      out[sg++] = g;
      st += static_cast<int64_t>(group_tiles(g)) * m.nh;
    }
  if (tid == 0) {
    m.plan->tiles = all;
    m.plan->per = per_cta(all, ctas);
    m.plan->ngroups = n;
  }
}

// A position on the line: item (group, head chunk) with tiles [s, e).
struct Walk {
  const Group *group;
  int nh, gi, c;
  int64_t s, e;
  Group g;
  __device__ void seek(const Plan *plan, const Group *groups, int heads, int64_t u) {
    group = groups;
    nh = heads;
    int lo = 0, hi = plan->ngroups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (group[mid].start <= u) lo = mid; else hi = mid;
    }
    gi = lo;
    g = group[gi];
    const int tiles = group_tiles(g);
    c = static_cast<int>((u - g.start) / tiles);
    s = g.start + static_cast<int64_t>(c) * tiles;
    e = s + tiles;
  }
  __device__ void next() {
    if (++c == nh) {
      c = 0;
      g = group[++gi];
    }
    s = e;
    e = s + group_tiles(g);
  }
  // Heads of this chunk, and score columns in use.
  __device__ int heads(const MmaArgs &m) const { return min(m.hc, m.a.H - c * m.hc); }
  __device__ int columns(const MmaArgs &m) const { return g.ntok == 1 ? heads(m) : g.ntok * m.hc; }
};

struct Small {
  float red[4][64];
  float sum[64], ref[64], factor[64];
  int end[64], token[64];
  uint32_t valid[kMaxStages][2];  // bit per key
  int key[2][kTile];
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t s_full[2], s_empty[2], p_full, o_done, q_full, q_empty, issued;
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(Small) <= kSmall, "small shared arrays");

template <class E, int N, bool BOX>
__global__ void __launch_bounds__(threads_of(BOX), 1)
    latent_attend_mma_kernel(const __grid_constant__ MmaArgs m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const LatentArgs &a = m.a;
  const int64_t per = m.plan->per, total = m.plan->tiles;
  const int64_t u0 = min(blockIdx.x * per, total), u1 = min(u0 + per, total);
  if (u0 >= u1) return;
  const int n_tiles = static_cast<int>(u1 - u0);
  const Group *groups = m.group;

  const int stage_bytes = m.np * kPanel, q_panel = N * 128;
  const uint32_t base = smem_addr(smem);
  const uint32_t q_at = base + m.nst * stage_bytes, p_at = q_at + m.np * q_panel;
  unsigned char *p_ptr = smem + (p_at - base);
  Small &sm = *reinterpret_cast<Small *>(p_ptr + kPanel);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wps = 8 / m.nst;  // copies: producer warps per stage
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(bar(sm.full[s]), BOX ? 2 : wps * 32);
      mbar_init(bar(sm.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(sm.s_full[s]), 1);
      mbar_init(bar(sm.s_empty[s]), kSoftmax);
    }
    mbar_init(bar(sm.p_full), kSoftmax);
    mbar_init(bar(sm.o_done), 1);
    mbar_init(bar(sm.issued), 1);
    mbar_init(bar(sm.q_full), query_threads(BOX));
    mbar_init(bar(sm.q_empty), 1);
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4) tmem_alloc(smem_addr(&sm.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, o_at = tmem + 2 * N;

  if constexpr (!BOX) {  // 128 x 200 + 384 x 104 registers = 512 x 128 at launch
    if (warp < 4) regs_raise<200>(); else regs_lower<104>();
  }
  if (warp < 4) {
    // ------------------------------------------------------- softmax, results
    constexpr int C = N / 2;  // columns per thread: [half C, half C + C) of key kk
    const int kk = warp * 16 + (lane & 15), half = lane >> 4, c0 = half * C;
    Walk w;
    w.seek(m.plan, groups, m.nh, u0);
    int64_t u = u0;
    int i = 0, stage = 0, use = 0;  // tile of this CTA, its stage, the stage's use
    while (u < u1) {
      const int64_t stop = min(w.e, u1);
      const int ncol = w.columns(m);
      // Per column, the token and the end below which it sees every key.  A
      // group of one token without a tree needs no mask: keys past its end
      // come as skipped rows.
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        const int t = w.g.t0 + min(n / m.hc, w.g.ntok - 1);
        const bool masked = a.rows == nullptr && (w.g.ntok > 1 || a.tree != nullptr) && n < ncol;
        sm.token[n] = t;
        sm.end[n] = masked ? max(a.row_ends[t], 0) : INT32_MAX;
      }
      named_sync(1, kSoftmax);
      int low = INT32_MAX;
#pragma unroll
      for (int x = 0; x < C; ++x) low = min(low, sm.end[c0 + x]);
      float l[C], ref[C];
#pragma unroll
      for (int x = 0; x < C; ++x) l[x] = 0.f, ref[x] = kUnset;
      const bool whole = u == w.s && stop == w.e;
      const int slot = u == w.s ? 1 : 0;
      bool first = true;
      for (; u < stop; ++u, ++i) {
        mbar_wait(bar(sm.s_full[i & 1]), (i >> 1) & 1, dead);
        mbar_wait(bar(sm.full[stage]), use & 1, dead);  // the stage's valid flags
        __syncwarp();
        tc_fence_after();
        uint32_t raw[C];
        tmem_ld_half<C>(raw, tmem + (i & 1) * N + (static_cast<uint32_t>(warp * 32) << 16));
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bar(sm.s_empty[i & 1]));
        const int j = static_cast<int>(u - w.s) * kTile + kk;
        const bool live = (sm.valid[stage][kk >> 5] >> (kk & 31)) & 1;
        float s[C];
#pragma unroll
        for (int x = 0; x < C; ++x) s[x] = __uint_as_float(raw[x]) * a.scale_log2;
        if (!live || j >= low) {
          // Some column may not see this key.  A masked score that is not
          // finite may come from a key row that is not: such a row would turn
          // the column's 0 weight into NaN, so it is cleared; columns that do
          // see it keep their NaN weight.
          bool odd = false;
#pragma unroll
          for (int x = 0; x < C; ++x) {
            const int end = sm.end[c0 + x];
            if (!live ||
                (j >= end && !(a.tree != nullptr && tree_bit(a, sm.token[c0 + x], j - end)))) {
              odd |= !(fabsf(s[x]) < INFINITY);
              s[x] = -INFINITY;
            }
          }
          if (odd) {
            unsigned char *row = smem + stage * stage_bytes + kk * 128;
            bool bad = false;
            for (int ch = 0; ch * 8 < a.dl; ++ch) {
              Pack8<E> v;
              v.u = *reinterpret_cast<const uint4 *>(row + (ch >> 3) * kPanel + (((ch & 7) ^ (kk & 7)) << 4));
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = Elem<E>::to2(v.h[y]);
                bad |= !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
              }
            }
            if (bad)
              for (int ch = 0; ch * 8 < a.dl; ++ch)
                *reinterpret_cast<uint4 *>(row + (ch >> 3) * kPanel + (((ch & 7) ^ (kk & 7)) << 4)) =
                    make_uint4(0, 0, 0, 0);
          }
        }
        bool pass = first;
#pragma unroll
        for (int x = 0; x < C; ++x) pass |= s[x] - ref[x] > kLag;
        if (named_any(1, kSoftmax, pass)) {
          // Move the references to the running maxima.
#pragma unroll
          for (int x = 0; x < C; ++x) {
            float mx = s[x];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
            if ((lane & 15) == 0) sm.red[warp][c0 + x] = mx;
          }
          named_sync(1, kSoftmax);
#pragma unroll
          for (int x = 0; x < C; ++x) {
            const int n = c0 + x;
            const float now = fmaxf(fmaxf(fmaxf(sm.red[0][n], sm.red[1][n]),
                                          fmaxf(sm.red[2][n], sm.red[3][n])), ref[x]);
            const float f = exp2_fast(ref[x] - now);
            l[x] *= f;
            ref[x] = now;
            if (warp == 0 && (lane & 15) == 0) sm.factor[n] = f, sm.ref[n] = now;
          }
          named_sync(1, kSoftmax);
          if (!first) {
            mbar_wait(bar(sm.o_done), (i - 1) & 1, dead);
            __syncwarp();
            tc_fence_after();
            for (int col = 0; col < m.nb * N; col += 16) {
              const uint32_t at = o_at + col + (static_cast<uint32_t>(warp * 32) << 16);
              uint32_t o[16];
              tmem_ld16(o, at);
              tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y)
                o[y] = __float_as_uint(__uint_as_float(o[y]) * sm.factor[(col & (N - 1)) + y]);
              tmem_st16(at, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        Pack8<E> p[C / 8];
#pragma unroll
        for (int x = 0; x < C; x += 2) {
          const float p0 = exp2_fast(s[x] - ref[x]), p1 = exp2_fast(s[x + 1] - ref[x + 1]);
          l[x] += p0;
          l[x + 1] += p1;
          p[x / 8].h[(x % 8) / 2] = Elem<E>::from2(p0, p1);
        }
        if (i > 0) mbar_wait(bar(sm.o_done), (i - 1) & 1, dead);  // P is free
#pragma unroll
        for (int x = 0; x < C / 8; ++x) {
          const int ch = half * (C / 8) + x;
          *reinterpret_cast<uint4 *>(p_ptr + kk * 128 + ((ch ^ (kk & 7)) << 4)) = p[x].u;
        }
        fence_async_shared();
        mbar_arrive(bar(sm.p_full));
        first = false;
        if (++stage == m.nst) stage = 0, ++use;
      }
      // Sums over the keys, then O.
#pragma unroll
      for (int x = 0; x < C; ++x) {
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[x] += __shfl_xor_sync(~0u, l[x], d);
        if ((lane & 15) == 0) sm.red[warp][c0 + x] = l[x];
      }
      named_sync(1, kSoftmax);
      float *part = m.parts + (blockIdx.x * 2 + slot) * m.part_stride;
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        const float sum = sm.red[0][n] + sm.red[1][n] + sm.red[2][n] + sm.red[3][n];
        if (whole) {
          sm.sum[n] = sum == 0.f ? 0.f : 1.f / sum;
          if (a.lse != nullptr && n < ncol)
            a.lse[static_cast<int64_t>(sm.token[n]) * a.H + w.c * m.hc + n % m.hc] =
                sum == 0.f ? -INFINITY : (sm.ref[n] + log2f(sum)) * kLn2;
        } else {
          part[static_cast<int64_t>(N) * a.dl + n] = sm.ref[n];
          part[static_cast<int64_t>(N) * a.dl + N + n] = sum;
        }
      }
      named_sync(1, kSoftmax);
      mbar_wait(bar(sm.o_done), (i - 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
      for (int col = 0; col < m.nb * N; col += 16) {
        const int n0 = col & (N - 1), dim = (col / N) * 128 + warp * 32 + lane;
        if (n0 >= ncol) continue;
        uint32_t o[16];
        tmem_ld16(o, o_at + col + (static_cast<uint32_t>(warp * 32) << 16));
        tmem_wait_ld();
        if (whole) {
          // Lanes of a pair swap so that each stores two columns of one head.
#pragma unroll
          for (int y = 0; y < 16; y += 2) {
            const float x0 = __uint_as_float(o[y]) * sm.sum[n0 + y];
            const float x1 = __uint_as_float(o[y + 1]) * sm.sum[n0 + y + 1];
            const float got = __shfl_xor_sync(~0u, (lane & 1) ? x0 : x1, 1);
            const int n = n0 + y + (lane & 1), d = dim & ~1;
            const float lo = (lane & 1) ? got : x0, hi = (lane & 1) ? x1 : got;
            if (n < ncol) {
              E *out = static_cast<E *>(a.out) + sm.token[n] * a.ld_out_t +
                       (w.c * m.hc + n % m.hc) * a.ld_out_h + d;
              if (m.out_vec) {
                if (d < a.dl) *reinterpret_cast<typename Elem<E>::T2 *>(out) = Elem<E>::from2(lo, hi);
              } else {
                if (d < a.dl) out[0] = Elem<E>::from(lo);
                if (d + 1 < a.dl) out[1] = Elem<E>::from(hi);
              }
            }
          }
        } else if (dim < a.dl) {
#pragma unroll
          for (int y = 0; y < 16; ++y)
            part[static_cast<int64_t>(n0 + y) * a.dl + dim] = __uint_as_float(o[y]);
        }
      }
      tc_fence_before();
      named_sync(1, kSoftmax);  // the per-column arrays are free
      if (u < u1) w.next();
    }
  } else if (warp == 4) {
    // -------------------------------------------------------------- MMA issue
    const uint32_t leader = elect_leader();
    constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
    constexpr uint32_t dq = mma_desc(bf16, false, false, kTile, N);
    constexpr uint32_t dp = mma_desc(bf16, true, true, 128, N);
    const int ksteps = (a.D + 15) / 16;
    // Descriptors hold addresses in units of 16 bytes: steps are added to them.
    const uint64_t k_desc = tile_desc(base, 16, 1024), q_desc = tile_desc(q_at, 16, 1024);
    const uint64_t v_desc = tile_desc(base, kPanel, 1024), p_desc = tile_desc(p_at, kPanel, 1024);
    Walk wq, wp;
    wq.seek(m.plan, groups, m.nh, u0);
    wp = wq;
    int iq = 0, ip = 0, q_stage = 0, q_use = 0, p_stage = 0, seg = 0;
    bool q_first = true, p_first = true;
    long long t0 = clock64();
    while (ip < n_tiles) {
      bool moved = false;
      if (iq < n_tiles && warp_poll(bar(sm.full[q_stage]), q_use & 1) &&
          (iq < 2 || warp_poll(bar(sm.s_empty[iq & 1]), ((iq >> 1) - 1) & 1)) &&
          (!q_first || warp_poll(bar(sm.q_full), seg & 1))) {
        tc_fence_after();
        uint64_t kd = k_desc + ((q_stage * stage_bytes) >> 4), qd = q_desc;
        const uint32_t s_at = tmem + (iq & 1) * N;
        int ks = 0;
        for (; ks + 4 <= ksteps; ks += 4, kd += kPanel >> 4, qd += q_panel >> 4) {
          mma_ss(leader, s_at, kd, qd, dq, ks > 0);
          mma_ss(leader, s_at, kd + 2, qd + 2, dq, true);
          mma_ss(leader, s_at, kd + 4, qd + 4, dq, true);
          mma_ss(leader, s_at, kd + 6, qd + 6, dq, true);
        }
        for (; ks < ksteps; ++ks, kd += 2, qd += 2) mma_ss(leader, s_at, kd, qd, dq, ks > 0);
        tc_commit(leader, bar(sm.s_full[iq & 1]));
        q_first = u0 + iq + 1 == wq.e;
        if (q_first) {
          tc_commit(leader, bar(sm.q_empty));
          ++seg;
          if (iq + 1 < n_tiles) wq.next();
        }
        ++iq;
        if (++q_stage == m.nst) q_stage = 0, ++q_use;
        moved = true;
      }
      if (ip < iq && warp_poll(bar(sm.p_full), ip & 1)) {
        tc_fence_after();
        uint64_t vd = v_desc + ((p_stage * stage_bytes) >> 4);
        for (int b = 0; b < m.nb; ++b, vd += (2 * kPanel) >> 4) {
          mma_ss(leader, o_at + b * N, vd, p_desc, dp, !p_first);
          mma_ss(leader, o_at + b * N, vd + 128, p_desc + 128, dp, true);
          mma_ss(leader, o_at + b * N, vd + 256, p_desc + 256, dp, true);
          mma_ss(leader, o_at + b * N, vd + 384, p_desc + 384, dp, true);
        }
        tc_commit(leader, bar(sm.empty[p_stage]));
        tc_commit(leader, bar(sm.o_done));
        p_first = u0 + ip + 1 == wp.e;
        if (p_first && ip + 1 < n_tiles) wp.next();
        ++ip;
        if (++p_stage == m.nst) p_stage = 0;
        moved = true;
      }
      if (moved) {
        t0 = clock64();
      } else if (__any_sync(~0u, *dead != 0 || clock64() - t0 > kWaitClocks)) {
        *dead = 1;
        break;
      }
    }
    tc_commit(leader, bar(sm.issued));
    mbar_drain(bar(sm.issued), 0);
  } else if (BOX && warp < 7) {
    // --------------------------------------------------------------- key rows
    const int mine = warp - 5, panels = (m.np + 1 - mine) >> 1;  // mine, mine + 2, ...
    Walk w;
    w.seek(m.plan, groups, m.nh, u0);
    int2 row;  // this lane's keys: lane and lane + 32 of the tile
    auto rows_of = [&](int64_t u) {
      if (u >= w.e) w.next();
      const int j = static_cast<int>(u - w.s) * kTile + lane;
      row.x = j < w.g.extent ? static_cast<int>(key_row(a, w.g.t0, w.g.req, j)) : -1;
      row.y = j + 32 < w.g.extent ? static_cast<int>(key_row(a, w.g.t0, w.g.req, j + 32)) : -1;
    };
    rows_of(u0);
    int *key = sm.key[mine];
    const uint32_t leader = elect_leader();
    for (int i = 0, stage = 0, use = 0; i < n_tiles; ++i) {
      if (use > 0) mbar_wait(bar(sm.empty[stage]), (use - 1) & 1, dead);
      if (mine == 0) {
        const unsigned lo = __ballot_sync(~0u, row.x >= 0), hi = __ballot_sync(~0u, row.y >= 0);
        if (lane == 0) sm.valid[stage][0] = lo, sm.valid[stage][1] = hi;
      }
      key[lane] = max(row.x, 0);
      key[lane + 32] = max(row.y, 0);
      __syncwarp();
      const uint32_t full = bar(sm.full[stage]);
      if (lane == 0) mbar_expect(full, panels * kPanel);
      __syncwarp();
      const uint32_t dst = base + stage * stage_bytes + mine * kPanel;
      for (int r = 0; r < kTile; r += m.run) {
        const int first = key[r];
        for (int p = 0; p < panels; ++p)
          tma_box(leader, dst + p * 2 * kPanel + r * 128, &m.rows, (2 * p + mine) * 64, first, full);
      }
      if (i + 1 < n_tiles) rows_of(u0 + i + 1);
      if (++stage == m.nst) stage = 0, ++use;
    }
    for (int i = max(0, n_tiles - m.nst); i < n_tiles; ++i)
      mbar_drain(bar(sm.full[i % m.nst]), (i / m.nst) & 1);
  } else if (warp == 7 || (!BOX && warp < 8)) {
    // ---------------------------------------------------------------- queries
    constexpr int threads = query_threads(BOX);
    const int tid = static_cast<int>(threadIdx.x) - (256 - threads), chunks = m.np * 8;
    Walk w;
    w.seek(m.plan, groups, m.nh, u0);
    for (int seg = 0;; ++seg) {
      if (seg > 0) mbar_wait(bar(sm.q_empty), (seg - 1) & 1, dead);
      const int ncol = w.columns(m);
      for (int x = tid; x < N * chunks; x += threads) {
        const int n = x / chunks, ch = x - n * chunks, col = ch * 8;
        const int tok = n / m.hc;
        const bool live = n < ncol && col < a.D;
        const uint32_t dst = q_at + (ch >> 3) * q_panel + n * 128 + (((ch & 7) ^ (n & 7)) << 4);
        const E *src = static_cast<const E *>(a.q);
        if (live)
          src += static_cast<int64_t>(w.g.t0 + tok) * a.ld_q_t +
                 static_cast<int64_t>(w.c * m.hc + n - tok * m.hc) * a.ld_q_h + col;
        if (m.q_vec) {
          cp_async16(dst, src, live);
        } else {
          E v[8];
#pragma unroll
          for (int y = 0; y < 8; ++y) v[y] = live ? src[y] : Elem<E>::from(0.f);
          Pack8<E> pk;
#pragma unroll
          for (int y = 0; y < 4; ++y) pk.h[y].x = v[2 * y], pk.h[y].y = v[2 * y + 1];
          *reinterpret_cast<uint4 *>(smem + (dst - base)) = pk.u;
        }
      }
      cp_async_wait_all();
      fence_async_shared();
      mbar_arrive(bar(sm.q_full));
      if (w.e >= u1) break;
      w.next();
    }
  } else {
    // ---------------------------------------------------- key rows, by copies
    const int pw = warp - 8, stage = pw / wps, rows = kTile / wps, r0 = (pw - stage * wps) * rows;
    if (!BOX && stage < m.nst && stage < n_tiles) {
      Walk w;
      w.seek(m.plan, groups, m.nh, u0);
      auto row_of = [&](int64_t u) {
        while (u >= w.e) w.next();
        const int j = static_cast<int>(u - w.s) * kTile + r0 + lane;
        return lane < rows && j < w.g.extent ? static_cast<int>(key_row(a, w.g.t0, w.g.req, j)) : -1;
      };
      const int ch = lane & 7, whole = a.D / 64, width = (a.D + 15) & ~15;
      const E *cache = static_cast<const E *>(a.cache);
      unsigned short *valid16 = reinterpret_cast<unsigned short *>(sm.valid[stage]);
      int row = row_of(u0 + stage);
      int use = 0;
      for (int i = stage; i < n_tiles; i += m.nst, ++use) {
        if (use > 0) mbar_wait(bar(sm.empty[stage]), (use - 1) & 1, dead);
        __syncwarp();
        const unsigned live_rows = __ballot_sync(~0u, row >= 0);
        if (lane == 0) {
          if (rows == 16) valid16[r0 / 16] = static_cast<unsigned short>(live_rows);
          else sm.valid[stage][r0 / 32] = live_rows;
        }
        for (int g = 0; g < rows; g += 4) {
          const int rr = g + (lane >> 3), r = r0 + rr;
          const int at = __shfl_sync(~0u, row, rr);
          const bool live = at >= 0;
          const E *src = cache + (live ? at : 0) * a.ld_cache + ch * 8;
          uint32_t dst = base + stage * stage_bytes + r * 128 + ((ch ^ (r & 7)) << 4);
#pragma unroll 4
          for (int p = 0; p < whole; ++p, src += 64, dst += kPanel) cp_async16(dst, src, live);
          const int col = whole * 64 + ch * 8;
          if (col < width) cp_async16(dst, col < a.D ? src : cache, live && col < a.D);
        }
        if (i + m.nst < n_tiles) row = row_of(u0 + i + m.nst);
        cp_async_wait_all();
        fence_async_shared();
        mbar_arrive(bar(sm.full[stage]));
      }
    }
  }
  __syncthreads();
  if (warp == 4) tmem_free(tmem, 512);
  if (threadIdx.x == 0 && *dead != 0 && a.status != nullptr)
    atomicOr(a.status, SATK_STATUS_STALLED);
}

// Joins the partial results of the group that CTA x leaves unfinished: weights
// 2^(m_i - max m) / sum, parts added in line order.
template <class E>
__global__ void __launch_bounds__(256) latent_join_kernel(const __grid_constant__ MmaArgs m, int N) {
  const LatentArgs &a = m.a;
  const int64_t per = m.plan->per, total = m.plan->tiles;
  const int64_t u0 = min(blockIdx.x * per, total), u1 = min(u0 + per, total);
  if (u0 >= u1 || u1 >= total) return;
  Walk w;
  w.seek(m.plan, m.group, m.nh, u1 - 1);
  if (w.s < u0 || w.e <= u1) return;
  const int n_parts = static_cast<int>((w.e - 1) / per) - blockIdx.x + 1;
  __shared__ float weight[256], red[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ncol = w.columns(m);
  auto part = [&](int i) {
    return m.parts + ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * m.part_stride;
  };
  for (int n = blockIdx.y; n < ncol; n += kCombineY) {
    float top = kUnset, sum = 0.f;
    const bool mine = static_cast<int>(threadIdx.x) < n_parts;
    if (mine) {
      const float *p = part(threadIdx.x) + static_cast<int64_t>(N) * a.dl;
      top = p[n];
      sum = p[N + n];
    }
    float mx = top;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, red[i]);
    const float f = mine ? exp2_fast(top - mx) : 0.f;
    weight[threadIdx.x] = f;
    float l = f * sum;
    if (!mine) l = 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(~0u, l, d);
    __syncthreads();
    if (lane == 0) red[warp] = l;
    __syncthreads();
    l = 0.f;
    for (int i = 0; i < 8; ++i) l += red[i];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = n / m.hc, t = w.g.t0 + tok, h = w.c * m.hc + n - tok * m.hc;
    E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h;
    for (int d = threadIdx.x; d < a.dl; d += 256) {
      float acc = 0.f;
#pragma unroll 4
      for (int i = 0; i < n_parts; ++i)
        acc = fmaf(weight[i], part(i)[static_cast<int64_t>(n) * a.dl + d], acc);
      out[d] = Elem<E>::from(acc * inv);
    }
    if (threadIdx.x == 0 && a.lse != nullptr)
      a.lse[static_cast<int64_t>(t) * a.H + h] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
    __syncthreads();
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n < 256 ? n : 256;
}

int columns_for(int hc, int tpg) {
  const int n = hc * tpg;
  return n <= 16 ? 16 : n <= 32 ? 32 : 64;
}

size_t group_bytes() { return (sizeof(Plan) + 15) / 16 * 16 + sizeof(Group) * kMaxTokens; }

template <class E, int N, bool BOX>
int launch(const MmaArgs &m, int ctas, int smem, cudaStream_t stream) {
  if (!allow_smem(latent_attend_mma_kernel<E, N, BOX>, smem)) return SATK_ECUDA;
  latent_attend_mma_kernel<E, N, BOX><<<ctas, threads_of(BOX), smem, stream>>>(m);
  latent_join_kernel<E><<<dim3(ctas, kCombineY), 256, 0, stream>>>(m, N);
  return launch_status();
}

template <class E, bool BOX>
int launch_columns(const MmaArgs &m, int N, int ctas, int smem, cudaStream_t stream) {
  return N == 16   ? launch<E, 16, BOX>(m, ctas, smem, stream)
         : N == 32 ? launch<E, 32, BOX>(m, ctas, smem, stream)
                   : launch<E, 64, BOX>(m, ctas, smem, stream);
}

template <class E>
int launch_all(const MmaArgs &m, int N, int ctas, int smem, cudaStream_t stream) {
  return m.run > 1 ? launch_columns<E, true>(m, N, ctas, smem, stream)
                   : launch_columns<E, false>(m, N, ctas, smem, stream);
}

}  // namespace

bool latent_attend_mma_fits(const LatentArgs &a) {
  return a.D % 8 == 0 && a.ld_cache % 8 == 0 && aligned16(a.cache) && a.cache_rows > 0 &&
         a.cache_rows <= INT32_MAX;
}

size_t latent_attend_mma_workspace(int H, int dl) {
  (void)H;
  const int ctas = sm_count();
  return group_bytes() + sizeof(float) * 2 * ctas * (64 * static_cast<size_t>(dl) + 128);
}

int latent_attend_mma(const LatentArgs &args, int dtype, int tokens_per_request, void *workspace,
                      cudaStream_t stream) {
  const int ctas = sm_count();
  if (ctas == 0) return SATK_ECUDA;
  MmaArgs m;
  m.a = args;
  m.nh = (args.H + 63) / 64;
  m.hc = (args.H + m.nh - 1) / m.nh;
  const int room = 64 / m.hc;
  m.tpg = tokens_per_request < room ? (tokens_per_request < 1 ? 1 : tokens_per_request) : room;
  const int N = columns_for(m.hc, m.tpg);
  m.tpg = N / m.hc < m.tpg ? N / m.hc : m.tpg;
  m.np = (args.D + 63) / 64;
  m.nb = (args.dl + 127) / 128;
  m.part_stride = static_cast<int64_t>(N) * args.dl + 2 * N;
  m.plan = static_cast<Plan *>(workspace);
  const int fixed = m.np * N * 128 + kPanel + kSmall, limit = 227 * 1024;
  m.nst = (limit - fixed) / (m.np * kPanel);
  if (m.nst > kMaxStages) m.nst = kMaxStages;
  const int smem = fixed + m.nst * m.np * kPanel;
  m.q_vec = aligned16(args.q) && (args.T == 1 || args.ld_q_t % 8 == 0) &&
            (args.H == 1 || args.ld_q_h % 8 == 0);
  m.out_vec = (reinterpret_cast<uintptr_t>(args.out) & 3u) == 0 && args.dl % 2 == 0 &&
              (args.T == 1 || args.ld_out_t % 2 == 0) && (args.H == 1 || args.ld_out_h % 2 == 0);
  // Rows that consecutive keys of a tile share in one block (a run is in the
  // cache as a whole, or from its first key on is not).
  m.run = 1;
  if (args.rows == nullptr && args.stride_rows >= args.block_size) {
    while (m.run < kTile && args.block_size % (2 * m.run) == 0) m.run *= 2;
    if (m.run < 8) m.run = 1;
  }
  if (m.run > 1 &&
      !tensor_map_16bit(&m.rows, dtype == SATK_BF16, args.cache, args.cache_rows, args.D,
                        args.ld_cache, m.run))
    return SATK_ECUDA;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  m.group = reinterpret_cast<Group *>(ws + (sizeof(Plan) + 15) / 16 * 16);
  m.parts = reinterpret_cast<float *>(ws + group_bytes());
  for (int t = 0; t < args.T; t += kMaxTokens) {
    LatentArgs &a = m.a;
    a = args;
    a.T = args.T - t < kMaxTokens ? args.T - t : kMaxTokens;
    a.q = static_cast<const uint16_t *>(args.q) + t * args.ld_q_t;
    a.out = static_cast<uint16_t *>(args.out) + t * args.ld_out_t;
    if (args.lse != nullptr) a.lse = args.lse + static_cast<int64_t>(t) * args.H;
    if (args.rows != nullptr) {
      a.rows = args.rows + t * args.ld_rows;
      if (args.counts != nullptr) a.counts = args.counts + t;
    } else {
      a.req_id = args.req_id + t;
      a.row_ends = args.row_ends + t;
      if (args.tree != nullptr) a.tree = args.tree + static_cast<int64_t>(t) * args.tree_words;
    }
    latent_plan_kernel<<<1, 1024, 0, stream>>>(m, ctas);
    const int rc = dtype == SATK_BF16 ? launch_all<__nv_bfloat16>(m, N, ctas, smem, stream)
                                      : launch_all<__half>(m, N, ctas, smem, stream);
    if (rc != SATK_OK) return rc;
  }
  return SATK_OK;
}

}  // namespace satk
