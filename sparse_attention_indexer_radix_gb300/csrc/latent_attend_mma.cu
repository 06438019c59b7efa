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
// The weights P are rounded to the cache's type, because both operands of a
// product have one type and the values are the cache's: each is off by half a
// step of itself at most (bf16 2^-8, fp16 2^-11), the output by that share of
// sum p |v|, as much as its own rounding may be.  l sums them before the
// rounding, so the lse is not touched; statistics, sums, O and partial results
// are fp32.  In fp16 weights below 2^-25 vanish next to a largest of 1 to 2^8.
//
// Key rows reach shared memory in two ways, each its own instantiation:
//  - BOX, where pages give runs of 8 or more keys that lie together: TMA boxes
//    of a run x 64 columns.  256 threads: warps 0-3 softmax and results, warp 4
//    issues the MMAs, warps 5-6 the boxes, warp 7 brings the queries.
//  - else (selected rows, tiny pages): 16-byte asynchronous copies by eight
//    warps, each stage filled by its own.  512 threads: warps 0-3 and 4 as above, 5-7 queries, 8-15 keys.
//    (Random rows of 1088 bytes, nothing else running: these copies 6.3 TB/s,
//    TMA's gather of four rows a request 5.0, bulk copies of a row 3.7.)
// A stage is handed over in two halves of its columns: the scores of the first
// columns begin while the others arrive, and the first columns' values are
// given back while the others' products run.
//
// A row that is skipped or not in the cache is masked; if what was read in its
// place is not finite, the softmax role clears it in the tile.
//
// Split: the tiles of all groups form one line that is cut into equal pieces,
// one per SM (kItemTiles more for each group, for its queries and results); a
// group cut across SMs leaves unnormalised partial results in the
// workspace that a second kernel joins in a fixed order.  Up to kInline tokens
// every CTA works out the line for itself; a kernel before does it for more.
//
// Bound and measured: 643 thousand rows of 448 columns, 32 heads (576 MB): 109 us
// with the join, 5.3 TB/s; 128 x 2048 selected rows of 544 columns, 64 heads (285
// MB): 84 us, 3.4 TB/s.  A tile's chain (load, scores, softmax, values) is what
// two or three stages have to hide: of 227 KB, 64 heads' queries of 544 columns
// take 72, and two stages of 72 remain.
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
constexpr int kInline = 512;             // tokens up to which CTAs plan for themselves
constexpr int kJoinY = 8;                // CTAs that share a join, one warp a column
constexpr int kItemTiles = 3;            // tiles that a group's own costs are worth
constexpr int kMinTiles = 2;             // tiles per SM below which no group is cut
constexpr float kLag = 8.f;              // log2 by which scores may pass m_n

// One group: its tokens, the keys any of them may see, and where its tiles
// (nh head chunks after each other) start on the line.
struct Group {
  int64_t start;
  int t0, ntok, extent, req;
};

struct Plan {
  int64_t tiles, per;  // on the line, per CTA
  int ngroups;
  int whole;           // one item (group, head chunk) per CTA: nothing is cut
  int pad[2];
  __device__ Group *groups() { return reinterpret_cast<Group *>(this + 1); }
};
constexpr size_t plan_bytes(int groups) { return (sizeof(Plan) + sizeof(Group) * groups + 15) / 16 * 16; }

struct MmaArgs {
  LatentArgs a;
  unsigned char *plans;  // one, or one per CTA
  int4 *joins;           // per CTA: token, column count, first head, parts (0: none)
  int inline_plan;
  float *parts;
  __device__ Plan *plan(int cta) const {
    return reinterpret_cast<Plan *>(plans + (inline_plan ? cta * plan_bytes(kInline) : 0));
  }
  int nh, hc;    // head chunks and heads per chunk
  int tpg;       // tokens per group
  int columns;   // N
  int may_cut;   // 0: the sizes alone rule out that a group is cut
  int np, nst;   // 64-column panels of a key row, stages
  int np0;       // panels of a stage's first half (all of them: there is no second)
  int nb;        // 128-column blocks of a value
  int part_ld;   // a partial result: N rows of part_ld values, N references, N sums
  int64_t part_stride;
  int q_box, q_vec, out_vec;  // queries by TMA, by 16-byte copies; 8-byte stores
  int run;           // rows of a box: consecutive keys that share a block (1: copies)
  CUtensorMap rows;  // the cache, in boxes of 64 columns x run rows
  CUtensorMap q;     // the queries, in boxes of 64 columns x hc heads x tpg tokens
};

__device__ __forceinline__ int group_tiles(const Group &g) {
  return g.extent > 0 ? (g.extent + kTile - 1) / kTile : 1;
}

__device__ __forceinline__ int64_t per_cta(int64_t tiles, int ctas) {
  const int64_t per = (tiles + ctas - 1) / ctas;
  return per < kMinTiles ? kMinTiles : per;
}

// What cutting groups costs a CTA, in tiles: two partial results written (12.5 K
// cycles each for 64 columns x 512 values, where a tile takes 3.8 K) and the join
// of its share.  Where every item can have a CTA of its own and the longest is
// longer than an equal piece by no more than that, nothing is cut (128 tokens of
// 2048 rows, 64 heads: 87 us cut, 84 us whole).
__host__ __device__ __forceinline__ int cut_cost(int columns) { return 2 + 10 * columns / 64; }

struct PlanScratch {
  int64_t tiles[32];
  int groups[32], longest[32];
};

// Groups in token order, and the prefix sum of their tiles, by one CTA of up to
// 1024 threads.
__device__ void make_plan(const MmaArgs &m, int ctas, Plan *plan, PlanScratch &scratch) {
  const LatentArgs &a = m.a;
  int64_t *wt = scratch.tiles;
  int *wg = scratch.groups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int per = (a.T + threads - 1) / threads;
  const int b = min(tid * per, a.T), e = min(b + per, a.T);
  auto leader = [&](int t) {
    return m.tpg == 1 || t % m.tpg == 0 || a.req_id[t] != a.req_id[t - 1];
  };
  auto group = [&](int t) {
    Group g;
    g.start = 0;
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
  int groups = 0, longest = 0;
  for (int t = b; t < e; ++t)
    if (leader(t)) {
      g = group(t);
      tiles += static_cast<int64_t>(group_tiles(g) + kItemTiles) * m.nh;
      longest = max(longest, group_tiles(g) + kItemTiles);
      ++groups;
    }
  int64_t st = tiles;
  int sg = groups;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, st, d);
    const int y = __shfl_up_sync(~0u, sg, d);
    if (lane >= d) st += x, sg += y;
    longest = max(longest, __shfl_xor_sync(~0u, longest, d));
  }
  if (lane == 31) wt[warp] = st, wg[warp] = sg, scratch.longest[warp] = longest;
  __syncthreads();
  int64_t all = 0;
  int n = 0;
  for (int w = 0; w < threads / 32; ++w) {
    longest = max(longest, scratch.longest[w]);
    if (w < warp) st += wt[w], sg += wg[w];
    all += wt[w];
    n += wg[w];
  }
  st -= tiles;
  sg -= groups;
  Group *out = plan->groups();
  for (int t = b; t < e; ++t)
    if (leader(t)) {
      if (groups > 1) g = group(t);
      g.start = st;
      out[sg++] = g;
      st += static_cast<int64_t>(group_tiles(g) + kItemTiles) * m.nh;
    }
  if (tid == 0) {
    plan->tiles = all;
    plan->per = per_cta(all, ctas);
    plan->ngroups = n;
    plan->whole = static_cast<int64_t>(n) * m.nh <= ctas &&
                  longest <= plan->per + cut_cost(m.columns);
  }
}

__global__ void __launch_bounds__(1024) latent_plan_kernel(const __grid_constant__ MmaArgs m, int ctas) {
  __shared__ PlanScratch scratch;
  make_plan(m, ctas, m.plan(0), scratch);
}

// One CTA's piece of the line: `length` positions from u0 on.
struct Piece {
  const Group *group;
  int nh, length;
};

// The items (group, head chunk) of a piece, in order, with the tiles [k0, k1) of
// each that the piece covers.
struct Walk {
  int gi, c, k0, k1, s;  // s: where the item starts, counted from u0
  int t0, ntok, extent, req;
  __device__ void load(const Piece &piece) {
    const Group g = piece.group[gi];
    t0 = g.t0;
    ntok = g.ntok;
    extent = g.extent;
    req = g.req;
  }
  __device__ int tiles() const { return extent > 0 ? (extent + kTile - 1) / kTile : 1; }
  __device__ void start(const Piece &piece, const Plan *plan, int64_t u0) {
    int lo = 0, hi = plan->ngroups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (piece.group[mid].start <= u0) lo = mid; else hi = mid;
    }
    gi = lo;
    load(piece);
    const int64_t past = u0 - piece.group[gi].start;
    c = static_cast<int>(past / (tiles() + kItemTiles));
    s = static_cast<int>(static_cast<int64_t>(c) * (tiles() + kItemTiles) - past);
    cut(piece);
    if (done()) next(piece);
  }
  __device__ void cut(const Piece &piece) {
    k0 = max(-s, 0);
    k1 = min(piece.length - s, tiles());
  }
  __device__ bool done() const { return k0 >= k1; }
  __device__ void next(const Piece &piece) {
    s += tiles() + kItemTiles;
    if (s >= piece.length) {
      k0 = k1 = 0;
      return;
    }
    if (++c == piece.nh) {
      c = 0;
      ++gi;
      load(piece);
    }
    cut(piece);
  }
  // Heads of this chunk, and score columns in use.
  __device__ int heads(const MmaArgs &m) const { return min(m.hc, m.a.H - c * m.hc); }
  __device__ int columns(const MmaArgs &m) const { return ntok == 1 ? heads(m) : ntok * m.hc; }
};

// One tile after the other.
struct Cursor {
  Walk w;
  int k;
  __device__ explicit Cursor(const Walk &from) : w(from), k(from.k0) {}
  __device__ bool more() const { return k < w.k1; }
  __device__ bool first() const { return k == w.k0; }
  __device__ bool last() const { return k + 1 == w.k1; }
  __device__ void step(const Piece &piece) {
    if (++k == w.k1) {
      w.next(piece);
      k = w.k0;
    }
  }
};

// Four consecutive results, of which the first `left` exist.
template <class E>
__device__ __forceinline__ void store4(E *out, float4 v, int left, bool vec) {
  union {
    typename Elem<E>::T2 h[2];
    uint2 u;
  } p;
  p.h[0] = Elem<E>::from2(v.x, v.y);
  p.h[1] = Elem<E>::from2(v.z, v.w);
  if (vec) {  // rows are 8-byte aligned and a multiple of four long
    if (left > 0) *reinterpret_cast<uint2 *>(out) = p.u;
  } else {
    if (left > 0) out[0] = p.h[0].x;
    if (left > 1) out[1] = p.h[0].y;
    if (left > 2) out[2] = p.h[1].x;
    if (left > 3) out[3] = p.h[1].y;
  }
}

// A reduction over the 16 keys (lanes of a half warp) of C columns at once: each
// step halves the columns a lane still has.  Afterwards a lane's v[0 .. C / 16)
// (v[0] at least) are the columns from `first` on.
struct Maximum {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};
struct Sum {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
template <class Op, int HAVE, int D, int C>
__device__ __forceinline__ void reduce_keys(float (&v)[C], int lane, int &first) {
  if constexpr (D > 0) {
    if constexpr (HAVE > 1) {
      const bool upper = lane & D;
#pragma unroll
      for (int x = 0; x < HAVE / 2; ++x) {
        const float give = upper ? v[x] : v[x + HAVE / 2];
        const float keep = upper ? v[x + HAVE / 2] : v[x];
        v[x] = Op::of(keep, __shfl_xor_sync(~0u, give, D));
      }
      if (upper) first += HAVE / 2;
      reduce_keys<Op, HAVE / 2, D / 2>(v, lane, first);
    } else {
      v[0] = Op::of(v[0], __shfl_xor_sync(~0u, v[0], D));
      reduce_keys<Op, 1, D / 2>(v, lane, first);
    }
  }
}

struct Small {
  float red[4][64];
  float ref[64];
  float factor[64];  // of a rescaling; at a group's end 1 / sum
  int end[64], token[64];
  unsigned long long sees[64];  // of a tile's keys, per column; at a group's end the output's offset
  uint32_t valid[kMaxStages][2];  // bit per key
  uint64_t full[kMaxStages][2], empty[kMaxStages][2];
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
  Plan *const plan = m.plan(blockIdx.x);
  wait_for_previous_kernel();
  if (m.inline_plan) {
    make_plan(m, gridDim.x, plan, *reinterpret_cast<PlanScratch *>(smem));
    fence_async_shared();
    __syncthreads();
  }
  const int64_t per = plan->per, total = plan->tiles;
  int64_t u0 = min(blockIdx.x * per, total), u1 = min(u0 + per, total);
  if (plan->whole) {
    const int gi = blockIdx.x / m.nh;
    u0 = u1 = 0;
    if (gi < plan->ngroups) {
      const Group g = plan->groups()[gi];
      const int length = group_tiles(g) + kItemTiles;
      u0 = g.start + (blockIdx.x - gi * m.nh) * length;
      u1 = u0 + length;
    }
  }
  const Piece piece{plan->groups(), m.nh, static_cast<int>(u1 - u0)};
  Walk w;
  w.k0 = w.k1 = 0;
  if (u0 < u1) w.start(piece, plan, u0);
  if (w.done()) {
    if (threadIdx.x == 0) m.joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }

  const int stage_bytes = m.np * kPanel, q_panel = N * 128;
  const uint32_t base = smem_addr(smem);
  const uint32_t q_at = base + m.nst * stage_bytes, p_at = q_at + m.np * q_panel;
  unsigned char *p_ptr = smem + (p_at - base);
  Small &sm = *reinterpret_cast<Small *>(p_ptr + kPanel);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wps = 8 / m.nst;  // copies: warps per stage
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(sm.full[s][h]), BOX ? 1 : wps * 32);
        mbar_init(bar(sm.empty[s][h]), 1);
      }
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(sm.s_full[s]), 1);
      mbar_init(bar(sm.s_empty[s]), kSoftmax);
    }
    mbar_init(bar(sm.p_full), kSoftmax);
    mbar_init(bar(sm.o_done), 1);
    mbar_init(bar(sm.issued), 1);
    mbar_init(bar(sm.q_full), m.q_box ? 1 : query_threads(BOX));
    mbar_init(bar(sm.q_empty), 1);
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4) tmem_alloc(smem_addr(&sm.tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, o_at = tmem + 2 * N;

  if constexpr (!BOX) {  // 128 x 216 + 384 x 96 registers, of 512 x 128 at launch
    if (warp < 4) regs_raise<216>(); else regs_lower<96>();
  }
  if (warp < 4) {
    // ------------------------------------------------------- softmax, results
    constexpr int C = N / 2;  // columns per thread: [half C, half C + C) of key kk
    const int kk = warp * 16 + (lane & 15), half = lane >> 4, c0 = half * C;
    int i = 0, stage = 0, use = 0;  // tile of this CTA, its stage, the stage's use
    for (; !w.done(); w.next(piece)) {
      const int ncol = w.columns(m);
      // Per column, the token and the end below which it sees every key.  A
      // group of one token without a tree needs no mask: keys past its end
      // come as skipped rows.
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        const int t = w.t0 + min(n / m.hc, w.ntok - 1);
        const bool masked = a.rows == nullptr && (w.ntok > 1 || a.tree != nullptr) && n < ncol;
        sm.token[n] = t;
        sm.end[n] = masked ? max(a.row_ends[t], 0) : INT32_MAX;
      }
      named_sync(1, kSoftmax);
      int low = INT32_MAX;
#pragma unroll
      for (int x = 0; x < N; ++x) low = min(low, sm.end[x]);
      float l[C], ref[C];
#pragma unroll
      for (int x = 0; x < C; ++x) l[x] = 0.f, ref[x] = kUnset;
      const bool whole = w.k0 == 0 && w.k1 == w.tiles();
      const int slot = w.k0 == 0 ? 1 : 0;
      // The CTA in which a group starts and does not end has it joined.
      if (threadIdx.x == 0) {
        const int end = w.s + w.tiles();  // that of its tiles
        m.joins[blockIdx.x] = make_int4(w.t0, ncol, w.c * m.hc,
                                        w.k0 == 0 && end > piece.length
                                            ? static_cast<int>((end - 1) / per) + 1 : 0);
      }
      // near: every reference is at most kFine; else the references are looked at
      // in every tile, which takes the exponents anew.
      bool first = true, near = false;
      for (int k = w.k0; k < w.k1; ++k, ++i) {
        mbar_wait(bar(sm.s_full[i & 1]), (i >> 1) & 1, dead);
        mbar_wait(bar(sm.full[stage][0]), use & 1, dead);  // the stage's valid flags
        __syncwarp();
        tc_fence_after();
        uint32_t raw[C];
        tmem_ld_half<C>(raw, tmem + (i & 1) * N + (static_cast<uint32_t>(warp * 32) << 16));
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(bar(sm.s_empty[i & 1]));
        const int j0 = k * kTile;
        if (j0 + kTile > low) {
          // Some column may not see some key: bit kk of sees[n].
          if (threadIdx.x < N) {
            const int n = threadIdx.x, past = j0 - sm.end[n];  // first key past the end
            unsigned long long sees = past >= 0 ? 0 : past <= -kTile ? ~0ull : ~0ull >> (kTile + past);
            if (a.tree != nullptr && n < ncol)
              for (int y = max(past >> 5, 0); y <= (past + kTile - 1) >> 5 && y < a.tree_words; ++y) {
                const unsigned long long bits = static_cast<uint32_t>(
                    a.tree[static_cast<int64_t>(sm.token[n]) * a.tree_words + y]);
                const int at = y * 32 - past;  // tile position of the word's first bit
                sees |= at >= 0 ? bits << at : bits >> -at;
              }
            sm.sees[n] = sees;
          }
          named_sync(1, kSoftmax);
        }
        const bool live = (sm.valid[stage][kk >> 5] >> (kk & 31)) & 1;
        float s[C];  // scores in log2, less their references
#pragma unroll
        for (int x = 0; x < C; ++x) s[x] = fmaf(__uint_as_float(raw[x]), a.scale_log2, -ref[x]);
        if (!live || j0 + kk >= low) {
          // Some column may not see this key.  A masked score that is not
          // finite may come from a key row that is not: such a row would turn
          // the column's 0 weight into NaN, so it is cleared; columns that do
          // see it keep their NaN weight.
          bool odd = false;
#pragma unroll
          for (int x = 0; x < C; ++x) {
            if (!live || !((sm.sees[c0 + x] >> kk) & 1)) {
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
        bool pass = !near;
#pragma unroll
        for (int x = 0; x < C; ++x) pass |= s[x] > kLag;
        if (named_any(1, kSoftmax, pass)) {
          // Move the references to the running maxima.
          {
            float mx[C];
#pragma unroll
            for (int x = 0; x < C; ++x)
              mx[x] = s[x] == -INFINITY ? s[x] : __fmul_rn(__uint_as_float(raw[x]), a.scale_log2);
            int at = c0;
            reduce_keys<Maximum, C, 8>(mx, lane, at);
#pragma unroll
            for (int x = 0; x < (C + 15) / 16; ++x) sm.red[warp][at + x] = mx[x];
          }
          named_sync(1, kSoftmax);
          near = true;
#pragma unroll
          for (int x = 0; x < C; x += 4) {
            float4 now = make_float4(ref[x], ref[x + 1], ref[x + 2], ref[x + 3]), f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float4 r = *reinterpret_cast<const float4 *>(&sm.red[y][c0 + x]);
              now.x = fmaxf(now.x, r.x);
              now.y = fmaxf(now.y, r.y);
              now.z = fmaxf(now.z, r.z);
              now.w = fmaxf(now.w, r.w);
            }
            auto move = [&](int at, float to) {
              const float factor = exp2_fast(ref[at] - to);
              l[at] *= factor;
              ref[at] = to;
              near &= fabsf(to) <= kFine || to == kUnset;
              if (s[at] != -INFINITY) s[at] = far_exponent(__uint_as_float(raw[at]), a.scale_log2, to);
              return factor;
            };
            f.x = move(x, now.x);
            f.y = move(x + 1, now.y);
            f.z = move(x + 2, now.z);
            f.w = move(x + 3, now.w);
            if (warp == 0 && (lane & 15) == 0) {
              *reinterpret_cast<float4 *>(&sm.factor[c0 + x]) = f;
              *reinterpret_cast<float4 *>(&sm.ref[c0 + x]) = now;
            }
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
          const float p0 = exp2_fast(s[x]), p1 = exp2_fast(s[x + 1]);
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
      {
        int at = c0;
        reduce_keys<Sum, C, 8>(l, lane, at);
#pragma unroll
        for (int x = 0; x < (C + 15) / 16; ++x) sm.red[warp][at + x] = l[x];
      }
      named_sync(1, kSoftmax);
      float *part = m.parts + (blockIdx.x * 2 + slot) * m.part_stride;
      float sum = 0.f;
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        sum = sm.red[0][n] + sm.red[1][n] + sm.red[2][n] + sm.red[3][n];
        if (whole) {
          sm.factor[n] = sum == 0.f ? 0.f : 1.f / sum;
          sm.sees[n] = sm.token[n] * a.ld_out_t + (w.c * m.hc + n % m.hc) * a.ld_out_h;
        }
      }
      named_sync(1, kSoftmax);
      mbar_wait(bar(sm.o_done), (i - 1) & 1, dead);
      __syncwarp();
      tc_fence_after();
      if (satk_stall_asked()) {  // debug build: after the last item nothing waits any more
        Walk after = w;
        after.next(piece);
        if (after.done()) *dead = 1;
      }
      if (*dead != 0) {
        // Some wait so far was given up: what there is may be anything.  The
        // statistics of a part carry the NaN into the join.
        sum = NAN;
        for (int n = lane; n < N; n += 32) sm.factor[n] = NAN;
        __syncwarp();
      }
      if (threadIdx.x < N) {
        const int n = threadIdx.x;
        if (!whole) {
          part[static_cast<int64_t>(N) * m.part_ld + n] = sm.ref[n];
          part[static_cast<int64_t>(N) * m.part_ld + N + n] = sum;
        } else if (a.lse != nullptr && n < ncol) {
          a.lse[static_cast<int64_t>(sm.token[n]) * a.H + w.c * m.hc + n % m.hc] =
              sum == 0.f ? -INFINITY : (sm.ref[n] + log2f(sum)) * kLn2;
        }
      }
      // A warp turns its 32 lanes x 16 columns through its quarter of the weights'
      // buffer, so that eight lanes store 32 consecutive values of a column
      // (stored as they come, a lane a value, 64 columns x 512 took 14 us).
      float *turn = reinterpret_cast<float *>(p_ptr) + warp * 512;
      const int y0 = lane >> 3, d0 = warp * 32 + (lane & 7) * 4;
      // Of the 16-column steps of each block only those with a column in use; the
      // next step's values are on their way while one is stored.
      const int steps = (ncol + 15) >> 4, total = m.nb * steps;
      int fetched = 0, fetch_at = 0;  // the step's column in tensor memory
      auto fetch = [&](uint32_t (&o)[16]) {
        tmem_ld16(o, o_at + fetch_at + (static_cast<uint32_t>(warp * 32) << 16));
        fetch_at += 16;
        if (++fetched == steps) fetched = 0, fetch_at += N - steps * 16;
      };
      int n0 = 0, d = d0;
      auto store = [&](const uint32_t (&o)[16]) {
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 16; ++y) turn[y * 32 + lane] = __uint_as_float(o[y]);
        __syncwarp();
        // All of shared memory's part first: stores to memory could alias it.
        float4 v[4];
        float f[4];
        long long off[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          v[y] = *reinterpret_cast<const float4 *>(turn + (4 * y + y0) * 32 + (lane & 7) * 4);
          f[y] = sm.factor[n0 + 4 * y + y0];
          off[y] = static_cast<long long>(sm.sees[n0 + 4 * y + y0]);
        }
        if (whole) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (n0 + 4 * y + y0 < ncol)
              store4<E>(static_cast<E *>(a.out) + off[y] + d,
                        make_float4(v[y].x * f[y], v[y].y * f[y], v[y].z * f[y], v[y].w * f[y]),
                        a.dl - d, m.out_vec);
        } else if (d < m.part_ld) {
          float *to = part + (n0 + y0) * m.part_ld + d;
#pragma unroll
          for (int y = 0; y < 4; ++y)
            __stcg(reinterpret_cast<float4 *>(to + 4 * y * m.part_ld), v[y]);
        }
        n0 += 16;
        if (n0 >= steps * 16) n0 = 0, d += 128;
      };
      uint32_t even[16], odd[16];
      fetch(even);
      for (int step = 0; step < total; step += 2) {
        tmem_wait_ld();
        if (step + 1 < total) fetch(odd);
        store(even);
        if (step + 1 < total) {
          tmem_wait_ld();
          if (step + 2 < total) fetch(even);
          store(odd);
        }
      }
      tc_fence_before();
      named_sync(1, kSoftmax);  // the per-column arrays are free
    }
  } else if (warp == 4) {
    // -------------------------------------------------------------- MMA issue
    if (elect_leader()) {
      constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
      constexpr uint32_t dq = mma_desc(bf16, false, false, kTile, N);
      constexpr uint32_t dp = mma_desc(bf16, true, true, 128, N);
      const int ksteps = (a.D + 15) / 16;
      // Descriptors hold addresses in units of 16 bytes: steps are added to them.
      const uint64_t k_desc = tile_desc(base, 16, 1024), q_desc = tile_desc(q_at, 16, 1024);
      const uint64_t v_desc = tile_desc(base, kPanel, 1024), p_desc = tile_desc(p_at, kPanel, 1024);
      Cursor cq(w), cp(w);  // the next tile of the scores and of the values
      const int ksteps0 = min(m.np0 * 4, ksteps), nb0 = m.np0 < m.np ? m.np0 / 2 : m.nb;
      int iq = 0, ip = 0, q_stage = 0, q_use = 0, p_stage = 0, seg = 0;
      bool q_half = false;  // the scores' first half is issued
      uint64_t kd = 0, qd = 0;
      auto scores = [&](int ks, int end) {
        const uint32_t s_at = tmem + (iq & 1) * N;
        for (; ks + 4 <= end; ks += 4, kd += kPanel >> 4, qd += q_panel >> 4) {
          mma_ss(s_at, kd, qd, dq, ks > 0);
          mma_ss(s_at, kd + 2, qd + 2, dq, true);
          mma_ss(s_at, kd + 4, qd + 4, dq, true);
          mma_ss(s_at, kd + 6, qd + 6, dq, true);
        }
        for (; ks < end; ++ks, kd += 2, qd += 2) mma_ss(s_at, kd, qd, dq, ks > 0);
      };
      bool moved = false;
      // A tile's values give its stage back, so they go between the two halves of
      // the next tile's scores (34 MMAs, 1450 cycles) as soon as they can.
      auto values = [&]() {
        if (ip < iq && mbar_poll(bar(sm.p_full), ip & 1)) {
          tc_fence_after();
          uint64_t vd = v_desc + ((p_stage * stage_bytes) >> 4);
          const bool more = !cp.first();
          for (int b = 0; b < m.nb; ++b, vd += (2 * kPanel) >> 4) {
            mma_ss(o_at + b * N, vd, p_desc, dp, more);
            mma_ss(o_at + b * N, vd + 128, p_desc + 128, dp, true);
            mma_ss(o_at + b * N, vd + 256, p_desc + 256, dp, true);
            mma_ss(o_at + b * N, vd + 384, p_desc + 384, dp, true);
            if (b + 1 == nb0) tc_commit(bar(sm.empty[p_stage][0]));
          }
          if (m.np0 < m.np) tc_commit(bar(sm.empty[p_stage][1]));
          tc_commit(bar(sm.o_done));
          cp.step(piece);
          ++ip;
          if (++p_stage == m.nst) p_stage = 0;
          moved = true;
        }
      };
      long long t0 = clock64();
      while (cp.more()) {
        moved = false;
        values();
        if (cq.more() && !q_half && mbar_poll(bar(sm.full[q_stage][0]), q_use & 1) &&
            (iq < 2 || mbar_poll(bar(sm.s_empty[iq & 1]), ((iq >> 1) - 1) & 1)) &&
            (!cq.first() || mbar_poll(bar(sm.q_full), seg & 1))) {
          tc_fence_after();
          kd = k_desc + ((q_stage * stage_bytes) >> 4);
          qd = q_desc;
          scores(0, ksteps0);
          q_half = moved = true;
        }
        values();
        if (q_half && (m.np0 == m.np || mbar_poll(bar(sm.full[q_stage][1]), q_use & 1))) {
          tc_fence_after();
          scores(ksteps0, ksteps);
          tc_commit(bar(sm.s_full[iq & 1]));
          if (cq.last()) {
            tc_commit(bar(sm.q_empty));
            ++seg;
          }
          cq.step(piece);
          ++iq;
          if (++q_stage == m.nst) q_stage = 0, ++q_use;
          q_half = false;
          moved = true;
        }
        if (moved) {
          t0 = clock64();
        } else if (*dead != 0 || clock64() - t0 > kWaitClocks) {
          *dead = 1;
          break;
        }
      }
      tc_commit(bar(sm.issued));
      mbar_drain(bar(sm.issued), 0);
    }
    __syncwarp();
  } else if (BOX && warp < 7) {
    // ------------------------------------------------------ key rows, in boxes
    // Warp 5 fills the stages' first halves, warp 6 the second ones.
    const int half = warp - 5, p0 = half == 0 ? 0 : m.np0, p1 = half == 0 ? m.np0 : m.np;
    if (p0 < p1) {
      // First rows of a tile's runs (m.run keys each), looked up for as many
      // tiles of the item at once as the warp has lanes for.
      const int runs = kTile / m.run, batch = 32 / runs;
      const uint32_t leader = elect_leader();
      Cursor c(w);
      int first_row = -1, k_batch = 0;
      int i = 0;
      for (int stage = 0, use = 0; c.more(); ++i) {
        if (c.first() || c.k == k_batch + batch) {
          k_batch = c.k;
          const int j = (k_batch + lane / runs) * kTile + lane % runs * m.run;
          first_row = j < c.w.extent && k_batch + lane / runs < c.w.k1
                          ? static_cast<int>(key_row(a, c.w.t0, c.w.req, j))
                          : -1;
        }
        const int lane0 = (c.k - k_batch) * runs;
        if (use > 0) mbar_wait(bar(sm.empty[stage][half]), (use - 1) & 1, dead);
        __syncwarp();
        if (half == 0) {
          bool live[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = lane + x * 32;
            const int64_t row = __shfl_sync(~0u, first_row, lane0 + key / m.run);
            live[x] = row >= 0 && c.k * kTile + key < c.w.extent;
            if (live[x] && row + key % m.run >= a.cache_rows) {
              live[x] = false;
              if (a.status != nullptr) atomicOr(a.status, SATK_STATUS_BAD_ROW);
            }
          }
          const unsigned lo = __ballot_sync(~0u, live[0]), hi = __ballot_sync(~0u, live[1]);
          if (lane == 0) sm.valid[stage][0] = lo, sm.valid[stage][1] = hi;
        }
        const uint32_t full = bar(sm.full[stage][half]);
        if (lane == 0) mbar_expect(full, (p1 - p0) * kPanel);
        __syncwarp();
        const uint32_t dst = base + stage * stage_bytes;
        for (int r = 0; r < runs; ++r) {
          const int first = max(__shfl_sync(~0u, first_row, lane0 + r), 0);
          for (int p = p0; p < p1; ++p)
            tma_box(leader, dst + p * kPanel + r * m.run * 128, &m.rows, p * 64, first, full);
        }
        __syncwarp();
        c.step(piece);
        if (++stage == m.nst) stage = 0, ++use;
      }
      for (int x = max(0, i - m.nst); x < i; ++x)
        mbar_drain(bar(sm.full[x % m.nst][half]), (x / m.nst) & 1);
    }
  } else if (warp == 7 || (!BOX && warp < 8)) {
    // ---------------------------------------------------------------- queries
    constexpr int threads = query_threads(BOX);
    const int tid = static_cast<int>(threadIdx.x) - (256 - threads), chunks = m.np * 8;
    if (m.q_box && warp == 7) {
      // Rows that no box writes stay zeros.
      const int used = m.hc * m.tpg, spare = N - used;
      for (int x = lane; x < spare * chunks; x += 32) {
        const int p = x / (spare * 8), y = x - p * spare * 8;
        *reinterpret_cast<uint4 *>(smem + (q_at - base) + p * q_panel + used * 128 + y * 16) =
            make_uint4(0, 0, 0, 0);
      }
      fence_async_shared();
      __syncwarp();
      const uint32_t leader = elect_leader();
      int seg = 0;
      for (;; ++seg) {
        if (seg > 0) mbar_wait(bar(sm.q_empty), (seg - 1) & 1, dead);
        __syncwarp();
        if (lane == 0) mbar_expect(bar(sm.q_full), used * m.np * 128);
        __syncwarp();
        for (int p = 0; p < m.np; ++p)
          tma_box3(leader, q_at + p * q_panel, &m.q, p * 64, w.c * m.hc, w.t0, bar(sm.q_full));
        w.next(piece);
        if (w.done()) break;
      }
      mbar_drain(bar(sm.q_full), seg & 1);
    }
    for (int seg = 0; !m.q_box; ++seg) {
      if (seg > 0) mbar_wait(bar(sm.q_empty), (seg - 1) & 1, dead);
      const int ncol = w.columns(m);
      for (int x = tid; x < N * chunks; x += threads) {
        const int n = x / chunks, ch = x - n * chunks, col = ch * 8;
        const int tok = n / m.hc;
        const bool live = n < ncol && col < a.D;
        const uint32_t dst = q_at + (ch >> 3) * q_panel + n * 128 + (((ch & 7) ^ (n & 7)) << 4);
        const E *src = static_cast<const E *>(a.q);
        if (live)
          src += static_cast<int64_t>(w.t0 + tok) * a.ld_q_t +
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
      w.next(piece);
      if (w.done()) break;
    }
  } else {
    // ---------------------------------------------------- key rows, by copies
    // A stage's warps share its rows.  While a tile's copies are in flight the
    // numbers of the stage's next rows are looked up, and when those arrive the
    // rows start on their way from HBM to L2: the stages alone do not hold what
    // HBM's latency takes.
    const int pw = warp - 8, stage = pw / wps, rows = kTile / wps, r0 = (pw - stage * wps) * rows;
    Cursor c(w);
    for (int i = 0; i < stage && c.more(); ++i) c.step(piece);
    if (!BOX && stage < m.nst && c.more()) {
      const int ch = lane & 7, width = (a.D + 15) & ~15;
      const E *cache = static_cast<const E *>(a.cache);
      int entry = 0, entry_j = -1;  // -1: no key
      auto look_up = [&]() {
        const int j = c.k * kTile + r0 + lane;
        entry_j = lane < rows && j < c.w.extent ? j : -1;
        if (entry_j >= 0) entry = key_entry(a, c.w.t0, c.w.req, j);
      };
      auto resolve = [&]() {
        return entry_j >= 0 ? static_cast<int>(entry_row(a, entry, entry_j)) : -1;
      };
      look_up();
      int row = resolve();
      // Panels [p0, p1) of this warp's rows, four rows x 128 bytes a request.
      auto copy = [&](int p0, int p1) {
        const int whole = min(a.D / 64 - p0, p1 - p0);
#pragma unroll 2
        for (int g = 0; g < rows; g += 4) {
          const int rr = g + (lane >> 3), r = r0 + rr;
          const int at = __shfl_sync(~0u, row, rr);
          const bool live = at >= 0;
          const E *src = cache + (live ? at : 0) * a.ld_cache + ch * 8 + p0 * 64;
          const uint32_t dst = base + stage * stage_bytes + p0 * kPanel + r * 128 + ((ch ^ (r & 7)) << 4);
#pragma unroll
          for (int p = 0; p < 5; ++p)
            if (p < whole) cp_async16(dst + p * kPanel, src + p * 64, live);
          const int col = (p0 + whole) * 64 + ch * 8;
          if (p0 + whole < p1 && col < width)
            cp_async16(dst + whole * kPanel, col < a.D ? src + whole * 64 : cache, live && col < a.D);
        }
      };
      for (int use = 0;; ++use) {
        if (use > 0) mbar_wait(bar(sm.empty[stage][0]), (use - 1) & 1, dead);
        __syncwarp();
        const unsigned live_rows = __ballot_sync(~0u, row >= 0);
        if (lane == 0) {
          if (rows == 16) reinterpret_cast<unsigned short *>(sm.valid[stage])[r0 / 16] = live_rows;
          else sm.valid[stage][r0 / 32] = live_rows;
        }
        copy(0, m.np0);
        cp_async_commit();
        if (m.np0 < m.np) {
          if (use > 0) mbar_wait(bar(sm.empty[stage][1]), (use - 1) & 1, dead);
          __syncwarp();
          copy(m.np0, m.np);
        }
        cp_async_commit();
        for (int i = 0; i < m.nst && c.more(); ++i) c.step(piece);
        const bool more = c.more();
        if (more) look_up();
        cp_async_wait_but_one();
        fence_async_shared();
        mbar_arrive(bar(sm.full[stage][0]));
        cp_async_wait_all();
        fence_async_shared();
        mbar_arrive(bar(sm.full[stage][1]));
        if (!more) break;
        row = resolve();
        for (int g = 0; g < rows; g += 4) {
          const int at = __shfl_sync(~0u, row, g + (lane >> 3));
          if (at >= 0)
            for (int col = ch * 64; col < a.D; col += 512)
              prefetch_line(cache + at * a.ld_cache + col);
        }
      }
    }
  }
  let_next_kernel_start();
  __syncthreads();
  if (warp == 4) tmem_free(tmem, 512);
  if (threadIdx.x == 0 && *dead != 0 && a.status != nullptr)
    atomicOr(a.status, SATK_STATUS_STALLED);
}

// Joins the partial results of the group that CTA x leaves unfinished: weights
// 2^(m_i - max m) / sum, parts added in line order.  One warp per column and 256
// of its values.
template <class E>
__global__ void __launch_bounds__(256, 6) latent_join_kernel(const __grid_constant__ MmaArgs m, int N) {
  wait_for_previous_kernel();
  const LatentArgs &a = m.a;
  const int4 join = m.joins[blockIdx.x];
  const int n_parts = join.w, ncol = join.y;
  if (n_parts == 0) return;
  const int lane = threadIdx.x & 31;
  auto part = [&](int i) {
    return m.parts + ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * m.part_stride;
  };
  const int per_column = (m.nb + 1) >> 1;
  for (int x = blockIdx.y * 8 + (threadIdx.x >> 5); x < ncol * per_column; x += kJoinY * 8) {
    const int n = x / per_column, d = (x - n * per_column) * 256 + lane * 4;
    const int64_t stat = static_cast<int64_t>(N) * m.part_ld + n;
    const int64_t value = static_cast<int64_t>(n) * m.part_ld + d;
    // Statistics of the first 32 parts and values of the first two, all in
    // flight together; few groups have more.
    float top = kUnset, sum = 0.f;
    if (lane < n_parts) {
      const float *p = part(lane) + stat;
      top = __ldcg(p);
      sum = __ldcg(p + N);
    }
    float4 v[2][2];
    auto load = [&](int i) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int z = 0; z < 2; ++z)
          v[y][z] = i + y < n_parts && d + z * 128 < m.part_ld
                        ? __ldcg(reinterpret_cast<const float4 *>(part(i + y) + value + z * 128))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float mx = top;
    for (int i = lane + 32; i < n_parts; i += 32) mx = fmaxf(mx, part(i)[stat]);
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, y));
    float f = exp2_fast(top - mx), l = f * sum;
    float4 acc[2] = {};
    for (int i = 0; i < n_parts; i += 2) {
      if (i > 0) {
        load(i);
        if ((i & 31) == 0) {
          f = 0.f;
          if (i + lane < n_parts) {
            const float *p = part(i + lane) + stat;
            f = exp2_fast(p[0] - mx);
            l += f * p[N];
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float fi = __shfl_sync(~0u, f, (i + y) & 31);
        if (i + y < n_parts) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            acc[z].x = fmaf(fi, v[y][z].x, acc[z].x);
            acc[z].y = fmaf(fi, v[y][z].y, acc[z].y);
            acc[z].z = fmaf(fi, v[y][z].z, acc[z].z);
            acc[z].w = fmaf(fi, v[y][z].w, acc[z].w);
          }
        }
      }
    }
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) l += __shfl_xor_sync(~0u, l, y);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = n / m.hc, t = join.x + tok, h = join.z + n - tok * m.hc;
    E *out = static_cast<E *>(a.out) + t * a.ld_out_t + h * a.ld_out_h + d;
#pragma unroll
    for (int z = 0; z < 2; ++z)
      store4<E>(out + z * 128, make_float4(acc[z].x * inv, acc[z].y * inv, acc[z].z * inv, acc[z].w * inv),
                a.dl - d - z * 128, m.out_vec);
    if (d == 0 && a.lse != nullptr)
      a.lse[static_cast<int64_t>(t) * a.H + h] = l == 0.f ? -INFINITY : (mx + log2f(l)) * kLn2;
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

size_t plans_bytes(int ctas) {
  const size_t one = plan_bytes(kMaxTokens), each = plan_bytes(kInline) * ctas;
  return one > each ? one : each;
}

// Launches after the stream's previous kernel without waiting for its end; the
// kernel waits for it itself.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int block, int smem, cudaStream_t stream,
                         A... args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(block);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

template <class E, int N, bool BOX>
int launch(const MmaArgs &m, int ctas, int smem, cudaStream_t stream) {
  if (!allow_smem(latent_attend_mma_kernel<E, N, BOX>, smem, kSmemLimit)) return SATK_ECUDA;
  int rc = SATK_OK;
  if (launch_early(latent_attend_mma_kernel<E, N, BOX>, dim3(ctas), threads_of(BOX), smem, stream,
                   m) != cudaSuccess ||
      (m.may_cut && launch_early(latent_join_kernel<E>, dim3(ctas, kJoinY), 256, 0, stream, m, N) !=
                        cudaSuccess))
    rc = SATK_ECUDA;
  return rc;
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
  return plans_bytes(ctas) + sizeof(int4) * ctas + sizeof(float) * 2 * ctas * (64 * static_cast<size_t>(dl + 3) + 128);
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
  m.columns = N;
  m.np = (args.D + 63) / 64;
  m.nb = (args.dl + 127) / 128;
  m.np0 = (m.nb + 1) / 2 * 2;
  if (m.np0 > m.np) m.np0 = m.np;
  m.part_ld = (args.dl + 3) & ~3;
  m.part_stride = static_cast<int64_t>(N) * m.part_ld + 2 * N;
  const int fixed = m.np * N * 128 + kPanel + kSmall;
  m.nst = (kSmemLimit - fixed) / (m.np * kPanel);
  if (m.nst > kMaxStages) m.nst = kMaxStages;
  const int smem = fixed + m.nst * m.np * kPanel;
  m.q_vec = aligned16(args.q) && (args.T == 1 || args.ld_q_t % 8 == 0) &&
            (args.H == 1 || args.ld_q_h % 8 == 0);
  m.q_box = m.q_vec;
  m.out_vec = (reinterpret_cast<uintptr_t>(args.out) & 7u) == 0 && args.dl % 4 == 0 &&
              (args.T == 1 || args.ld_out_t % 4 == 0) && (args.H == 1 || args.ld_out_h % 4 == 0);
  // Rows that consecutive keys of a tile share in one block (a run is in the
  // cache as a whole, or from its first key on is not).
  m.run = 1;
  if (args.rows == nullptr && args.stride_rows >= args.block_size) {
    while (m.run < kTile && args.block_size % (2 * m.run) == 0) m.run *= 2;
    if (m.run < 8) m.run = 1;
  }
  const bool bf16 = dtype == SATK_BF16;
  if (m.run > 1 && !tensor_map_16bit(&m.rows, bf16, args.cache, args.D, args.cache_rows,
                                     args.ld_cache, m.run))
    return SATK_ECUDA;
  m.plans = static_cast<unsigned char *>(workspace);
  m.joins = reinterpret_cast<int4 *>(m.plans + plans_bytes(ctas));
  m.parts = reinterpret_cast<float *>(m.joins + ctas);
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
    // Strides of dimensions of one are free: any multiple of 16 bytes.
    if (m.q_box && !tensor_map_16bit(&m.q, bf16, a.q, a.D, a.H, a.H == 1 ? 1024 : a.ld_q_h, m.hc,
                                     a.T, args.T == 1 ? 1024 : a.ld_q_t, m.tpg))
      m.q_box = 0;
    m.inline_plan = a.T <= kInline;
    // (per_cta() is kMinTiles at least, so this is make_plan()'s rule.)
    m.may_cut = a.rows == nullptr || static_cast<int64_t>(a.T) * m.nh > ctas ||
                (a.k + kTile - 1) / kTile + kItemTiles > kMinTiles + cut_cost(N);
    if (!m.inline_plan) latent_plan_kernel<<<1, 1024, 0, stream>>>(m, ctas);
    const int rc = dtype == SATK_BF16 ? launch_all<__nv_bfloat16>(m, N, ctas, smem, stream)
                                      : launch_all<__half>(m, N, ctas, smem, stream);
    if (rc != SATK_OK) return rc;
  }
  return SATK_OK;
}

}  // namespace satk
