// latent_weights_mma.cu -- attention weights over selected rows on the tensor cores.
//
// Per token and tile of 128 of its entries:
//   S[entry, head] = K[entry, :] . Q[head, :]      M = 128 entries, N heads
//   out[entry]     = 1/H sum_head exp(scale S - lse)
// The entries are the M side, so that what is summed, the heads, lies along the
// columns of tensor memory.  There is no maximum to look for: lse is known.
//
// The rows arrive in panels of 64 columns x 128 rows through one ring that holds as
// many panels as shared memory has room for; a panel's products start when it is
// there.  Four groups of two warps bring panels in turn, by 16-byte asynchronous
// copies or the TMA's gathers.  A unit of work is a token and a piece of its tiles,
// dealt out over persistent CTAs; the next unit's queries replace this one's a panel
// at a time, behind the last tile's products.
//
// Bounded by the ring: 512 tokens x 2048 rows of 544 columns, 64 heads, are 1.1 GB
// through shared memory: 154 us, 132 with warm caches (8.6 TB/s; 36 us of products
// at the bf16 rate).  Without the copies it takes 97, without the products 146.
#include <cuda.h>
#include <type_traits>

#include "latent_weights.cuh"
#include "satk_tcgen05.cuh"

namespace satk {
namespace {

constexpr int kRows = 128;             // entries of a tile
constexpr int kPanel = kRows * 128;    // bytes of 64 columns of a tile
constexpr int kThreads = 512;          // warps 0-3 sums, 4 MMAs, 5 queries, 8-15 rows
constexpr int kMaxWide = 9;            // panels of a row
constexpr int kMaxSlots = 12;
constexpr int kGroups = 4;             // of row warps
constexpr int kHeads = 128;            // of a chunk
constexpr int kUnitTiles = 4;          // tiles worth a load of queries

struct WeightsMma {
  WeightsArgs a;
  int panels, last_steps;    // steps of 16 columns of the last panel
  int slots, heads, chunks;  // heads of a chunk (a multiple of 16), chunks
  int tiles, pieces, per;    // tiles of k entries, pieces of a token's tiles, tiles of a piece
  int step_t, step_piece;    // from a CTA's unit to its next
  CUtensorMap q, rows;
};

struct Small {
  uint64_t full[kMaxSlots], empty[kMaxSlots], q_full[kMaxWide], q_empty[kMaxWide];
  uint64_t s_full[2], s_empty[2], issued;
  uint32_t tmem;
  int dead;
};

// A CTA's units in order: token t, piece of its tiles.  The next one's count is on
// its way while one is worked on.
struct Units {
  const WeightsMma &m;
  int t, piece, next_t, next_piece, count, next_count;
  __device__ __forceinline__ Units(const WeightsMma &m) : m(m) {
    next_t = static_cast<int>(blockIdx.x) / m.pieces;
    next_piece = static_cast<int>(blockIdx.x) - next_t * m.pieces;
    next_count = next_t < m.a.T ? entry_count(m.a, next_t) : 0;
    next();
  }
  __device__ __forceinline__ bool more() const { return t < m.a.T; }
  __device__ __forceinline__ void next() {
    t = next_t, piece = next_piece, count = next_count;
    if (t >= m.a.T) return;
    next_t += m.step_t;
    next_piece += m.step_piece;
    if (next_piece >= m.pieces) next_piece -= m.pieces, ++next_t;
    if (next_t < m.a.T) next_count = entry_count(m.a, next_t);
  }
  __device__ __forceinline__ int first() const { return piece * m.per; }
  __device__ __forceinline__ int last() const { return min(first() + m.per, m.tiles); }
  // tiles of the piece with an entry that counts
  __device__ __forceinline__ int tiles() const {
    return max(0, min(last(), (count + kRows - 1) / kRows) - first());
  }
};

template <int N>
__device__ __forceinline__ void cp_async_wait_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
using Const = std::integral_constant<int, N>;

// f(panels) with a constant.
template <class F>
__device__ __forceinline__ void with_panels(int panels, F f) {
  switch (panels) {
    case 1: return f(Const<1>());
    case 2: return f(Const<2>());
    case 3: return f(Const<3>());
    case 4: return f(Const<4>());
    case 5: return f(Const<5>());
    case 6: return f(Const<6>());
    case 7: return f(Const<7>());
    case 8: return f(Const<8>());
    default: return f(Const<9>());
  }
}

// DEPTH: panels that a group of row warps has in flight by copies; 0: by the TMA's
// gathers, as many as the ring holds.
template <class E, int DEPTH>
__global__ void __launch_bounds__(kThreads, 1) latent_weights_mma_kernel(const __grid_constant__ WeightsMma m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const WeightsArgs &a = m.a;
  const uint32_t base = smem_addr(smem);
  const int q_panel = m.heads * 128, ring_at = m.panels * q_panel;
  Small &sm = *reinterpret_cast<Small *>(smem + ring_at + m.slots * kPanel);
  volatile int *dead = &sm.dead;
  auto bar = [&](uint64_t &b) { return smem_addr(&b); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t buffer = m.heads, columns = m.heads <= 16 ? 32 : m.heads <= 32 ? 64 : m.heads <= 64 ? 128 : 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < m.slots; ++s) {
      mbar_init(bar(sm.full[s]), 2);
      mbar_init(bar(sm.empty[s]), 1);
    }
    for (int p = 0; p < m.panels; ++p) {
      mbar_init(bar(sm.q_full[p]), 1);
      mbar_init(bar(sm.q_empty[p]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(sm.s_full[b]), 1);
      mbar_init(bar(sm.s_empty[b]), 4);
    }
    mbar_init(bar(sm.issued), 1);
    sm.dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 4) tmem_alloc(smem_addr(&sm.tmem), columns);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < 4) {
    // --------------------------------------------------------------------- sums
    // A thread has two of every eight heads of four entries.
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float2 scale2 = make_float2(a.scale, a.scale), log2e2 = make_float2(kLog2e, kLog2e);
    const float share = 1.f / a.H;
    int done = 0;  // tiles so far
    for (Units w(m); w.more(); w.next()) {
      const int n = w.tiles();
      float *out = a.out + w.t * a.ld_out;
      for (int c = 0; n > 0 && c < m.chunks; ++c) {
        // -lse; a head that saw nothing, or that is not there, adds nothing
        float2 less[kHeads / 8];
#pragma unroll
        for (int j = 0; j < kHeads / 8; ++j) {
          const int h = c * m.heads + 8 * j + 2 * (lane & 3);
          const float *lse = a.lse + static_cast<int64_t>(w.t) * a.H + h;
          const float x = 8 * j < m.heads && h < a.H ? lse[0] : -INFINITY;
          const float y = 8 * j < m.heads && h + 1 < a.H ? lse[1] : -INFINITY;
          less[j] = make_float2(x == -INFINITY ? x : -x, y == -INFINITY ? y : -y);
        }
        // whether the next tile's entries count
        int row[4];
        auto look_up = [&](int i) {
          const int e = (w.first() + i) * kRows + warp * 32 + (lane >> 2);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            row[r] = e + 8 * r < w.count ? a.rows[w.t * a.ld_rows + e + 8 * r] : -1;
        };
        look_up(0);
        for (int i = 0; i < n; ++i, ++done) {
          const int b = done & 1;
          const int entry0 = (w.first() + i) * kRows + warp * 32 + (lane >> 2);
          bool live[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) live[r] = row[r] >= 0 && row[r] < a.cache_rows;
          if (i + 1 < n) look_up(i + 1);
          mbar_wait(bar(sm.s_full[b]), (done >> 1) & 1, dead);
          __syncwarp();
          tc_fence_after();
          float2 sum[4];
          auto add_up = [&](auto careful) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum[r] = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kHeads / 32; ++j) {
              if (32 * j >= m.heads) break;
              uint32_t s[32];
              const uint32_t at = tmem + b * buffer + 32 * j + lanes;
              if (32 * j + 32 <= m.heads) {
                tmem_ld_pairs(s, 0, at);
                tmem_ld_pairs(s, 16, at + (16u << 16));
              } else {
                tmem_ld_pairs_half(s, 0, at);
                tmem_ld_pairs_half(s, 16, at + (16u << 16));
#pragma unroll
                for (int x = 8; x < 16; ++x) s[x] = s[16 + x] = 0;
              }
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float2 l = less[4 * j + (x >> 1 & 3)];
                float2 e = __ffma2_rn(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
                                      scale2, l);
                asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.x));  // (as head_weight)
                asm("min.NaN.f32 %0, %0, 0f00000000;" : "+f"(e.y));
                e = __fmul2_rn(e, log2e2);
                e.x = exp2_fast(e.x);
                e.y = exp2_fast(e.y);
                if (careful.value != 0) {
                  if (l.x == -INFINITY) e.x = 0.f;
                  if (l.y == -INFINITY) e.y = 0.f;
                }
                const int r = (x >> 3) * 2 + (x & 1);
                sum[r] = __fadd2_rn(sum[r], e);
              }
            }
          };
          // A head that adds nothing has -inf for -lse, and so for every exponent but that
          // of a score that is NaN or infinite: where a NaN comes out, once more with a look
          // at each head.
          add_up(Const<0>());
          const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          const float check = all.x + all.y;  // (weights are at most 1: no infinity among them)
          if (__any_sync(~0u, check != check)) add_up(Const<1>());
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(sm.s_empty[b]));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float x = sum[r].x + sum[r].y;
            x += __shfl_xor_sync(~0u, x, 1);
            x += __shfl_xor_sync(~0u, x, 2);
            const int e = entry0 + 8 * r;
            if ((lane & 3) == 0 && e < a.k) {
              x = *dead != 0 ? NAN : live[r] ? x * share : 0.f;
              out[e] = c == 0 ? x : out[e] + x;
            }
          }
        }
      }
      // Entries behind the token's count.
      const int end = min(w.last() * kRows, a.k);
      for (int e = (w.first() + n) * kRows + threadIdx.x; e < end; e += kRows) out[e] = 0.f;
    }
    if (threadIdx.x == 0 && *dead != 0 && a.status != nullptr) atomicOr(a.status, SATK_STATUS_STALLED);
  } else if (warp == 4) {
    // ---------------------------------------------------------------- MMA issue
    if (elect_leader()) {
      const uint32_t desc = mma_desc(std::is_same<E, __nv_bfloat16>::value, false, false, kRows, m.heads);
      const uint32_t full = bar(sm.full[0]), empty = bar(sm.empty[0]), q_full = bar(sm.q_full[0]);
      const uint32_t q_empty = bar(sm.q_empty[0]), s_full = bar(sm.s_full[0]), s_empty = bar(sm.s_empty[0]);
      const uint32_t q_low = desc_low(base, 16), ring_low = desc_low(base + ring_at, 16);
      const uint32_t q_step = q_panel >> 4, slots = m.slots, last_steps = m.last_steps;
      uint32_t slot = 0, phase = 0, done = 0, loads = 0;
      with_panels(m.panels, [&](auto panels) {
        // One tile; the first of a unit waits for its queries, behind the last one's
        // products their places are free.
        auto tile = [&](auto first, bool last) {
          const uint32_t b = done & 1, d = tmem + b * buffer;
          mbar_wait(s_empty + 8 * b, (done >> 1 & 1) ^ 1, dead);
#pragma unroll
          for (int p = 0; p < panels.value; ++p) {
            if (first.value != 0) mbar_wait(q_full + 8 * p, loads & 1, dead);
            mbar_wait(full + 8 * slot, phase, dead);
            tc_fence_after();
            const uint32_t k = ring_low + slot * (kPanel >> 4), q = q_low + p * q_step;
            const bool whole = p < panels.value - 1;
            mma_ss_low(d, k, q, desc, p > 0);
            mma_ss_low_if(whole || last_steps > 1, d, k + 2, q + 2, desc);
            mma_ss_low_if(whole || last_steps > 2, d, k + 4, q + 4, desc);
            mma_ss_low_if(whole || last_steps > 3, d, k + 6, q + 6, desc);
            tc_commit(empty + 8 * slot);
            tc_commit_if(last, q_empty + 8 * p);
            const bool wrap = slot + 1 == slots;
            slot = wrap ? 0 : slot + 1;
            phase ^= wrap ? 1 : 0;
          }
          tc_commit(s_full + 8 * b);
          ++done;
        };
        for (Units w(m); w.more(); w.next()) {
          const int n = w.tiles();
          for (int c = 0; n > 0 && c < m.chunks; ++c, ++loads) {
            tile(Const<1>(), n == 1);
            for (int i = 1; i < n; ++i) tile(Const<0>(), i == n - 1);
          }
        }
      });
      tc_commit(bar(sm.issued));
      mbar_drain(bar(sm.issued), 0);
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------------ queries
    const uint32_t leader = elect_leader();
    int loads = 0;
    for (Units w(m); w.more(); w.next())
      for (int c = 0; w.tiles() > 0 && c < m.chunks; ++c, ++loads)
        for (int p = 0; p < m.panels; ++p) {
          if (loads > 0) mbar_wait(bar(sm.q_empty[p]), (loads - 1) & 1, dead);
          __syncwarp();
          if (lane == 0) mbar_expect(bar(sm.q_full[p]), q_panel);
          __syncwarp();
          tma_box3(leader, base + p * q_panel, &m.q, p * 64, c * m.heads, w.t, bar(sm.q_full[p]));
        }
    if (loads > 0)
      for (int p = 0; p < m.panels; ++p) mbar_drain(bar(sm.q_full[p]), (loads - 1) & 1);
  } else if (warp >= 8) {
    // --------------------------------------------------------------------- rows
    // Two warps share a panel, 64 rows each, four rows x 128 bytes an instruction;
    // four such groups take panels in turn, DEPTH of them in flight each.
    const int group = (warp - 8) >> 1, r0 = (warp & 1) * 64, ch = lane & 7;
    const E *cache = static_cast<const E *>(a.cache) + ch * 8;
    // (row r0 + 4 g + lane / 8; the swizzle repeats every eight rows)
    uint32_t dst[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int r = r0 + 4 * g + (lane >> 3);
      dst[g] = base + ring_at + r * 128 + ((ch ^ (r & 7)) << 4);
    }
    int slot = group % m.slots, around = group / m.slots, filled = 0, told = 0, told_slot = slot;
    int total = 0;  // panels of all groups
    auto advance = [&](int &at) {
      at += kGroups;
      const bool wrap = at >= m.slots;
      if (wrap) at -= m.slots;
      return wrap;
    };
    auto tell = [&]() {  // the oldest panel that has not been handed over
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.full[told_slot]));
      advance(told_slot);
      ++told;
    };
    Units w(m);
    int c = 0, i = 0, p = group;  // the next panel of the tile for this group
    while (w.more() && w.tiles() == 0) w.next();
    // A gather brings four rows x 128 bytes (a skipped entry gets row 0, which nothing
    // looks at): 7.0 TB/s at most, but nobody waits for it, so it is what a short ring
    // wants.
    constexpr bool gather = DEPTH == 0;
    int2 row = make_int2(-1, -1);  // of this lane: entries r0 + lane and r0 + 32 + lane
    int4 four = make_int4(0, 0, 0, 0);  // or four from r0 + 4 lane on
    auto look_up = [&]() {
      const int e = (w.first() + i) * kRows + r0;
      auto at = [&](int x) { return static_cast<int>(entry_row(a, w.t, x, w.count)); };
      if (!gather) row = make_int2(at(e + lane), at(e + lane + 32));
      else if (lane < 16)
        four = make_int4(max(at(e + 4 * lane), 0), max(at(e + 4 * lane + 1), 0),
                         max(at(e + 4 * lane + 2), 0), max(at(e + 4 * lane + 3), 0));
    };
    if (w.more()) look_up();
    while (w.more()) {
      const int2 now = row;
      const int4 now4 = four;
      // the next tile's rows are looked up while this one's are copied
      if (++i == w.tiles()) {
        i = 0;
        if (++c == m.chunks) {
          c = 0;
          do w.next();
          while (w.more() && w.tiles() == 0);
        }
      }
      if (w.more()) look_up();
      for (; p < m.panels; p += kGroups) {
        mbar_wait(bar(sm.empty[slot]), (around & 1) ^ 1, dead);
        __syncwarp();
        const uint32_t to = slot * kPanel;
        if (gather) {
          if (lane == 0) mbar_expect(bar(sm.full[slot]), kPanel / 2);
          __syncwarp();
          if (lane < 16)
            tma_gather4(base + ring_at + to + (r0 + 4 * lane) * 128, &m.rows, p * 64, now4, bar(sm.full[slot]));
        } else {
          const bool wide = p < m.panels - 1 || ch < 2 * m.last_steps;
#pragma unroll
          for (int g = 0; g < 16; ++g) {
            const int at = __shfl_sync(~0u, g < 8 ? now.x : now.y, (4 * g & 31) + (lane >> 3));
            const bool live = at >= 0;
            const E *src = cache + static_cast<int64_t>(live ? at : 0) * a.ld_cache + p * 64;
            if (wide) cp_async16(dst[g & 1] + to + (g >> 1) * 1024, src, live);
          }
          cp_async_commit();
          if (++filled >= DEPTH) {
            cp_async_wait_but<(DEPTH > 0 ? DEPTH - 1 : 0)>();
            tell();
          }
        }
        if (advance(slot)) ++around;
      }
      p -= m.panels;
      total += m.panels;
    }
    // The gathers of the ring's last round, whether anyone has waited for them or not.
    // (An earlier one's slot has had another panel since, and its phase is no longer
    // told from the next but one.)
    for (int x = group; gather && x < total; x += kGroups)
      if (x >= total - m.slots) mbar_drain(bar(sm.full[x % m.slots]), x / m.slots & 1);
    cp_async_wait_all();
    while (told < filled) tell();
  }
  __syncthreads();
  if (warp == 4) tmem_free(tmem, columns);
}

// Copies in flight: the oldest panel of a group that has not been handed over waits
// until one kGroups (DEPTH - 1) further on has found room.  512 tokens x 2048 rows of
// 544 columns, with warm caches: 64 heads (a ring of 9 panels) 131 us with copies two
// deep, 163 with gathers; 128 heads (a ring of 4) 192 with gathers, 284 with copies one
// deep.
constexpr int kDepth = 2;
static_assert(kMaxSlots >= kGroups, "a group's next slot is less than a round further");

bool plan(const WeightsArgs &a, WeightsMma &m, int &smem) {
  m.panels = (a.D + 63) / 64;
  m.last_steps = (a.D - (m.panels - 1) * 64) / 16;
  m.chunks = (a.H + kHeads - 1) / kHeads;
  m.heads = ((a.H + m.chunks - 1) / m.chunks + 15) & ~15;
  m.chunks = (a.H + m.heads - 1) / m.heads;
  const int q = m.panels * m.heads * 128;
  m.slots = (kSmemLimit - q - static_cast<int>(sizeof(Small))) / kPanel;
  if (m.slots > kMaxSlots) m.slots = kMaxSlots;
  smem = q + m.slots * kPanel + static_cast<int>(sizeof(Small));
  return m.slots >= kGroups;
}

template <class E, int DEPTH>
int launch(WeightsMma &m, int smem, cudaStream_t stream) {
  auto kernel = latent_weights_mma_kernel<E, DEPTH>;
  if (!allow_smem(kernel, smem, kSmemLimit)) return SATK_ECUDA;
  const int64_t ctas = resident_ctas(reinterpret_cast<const void *>(kernel), kThreads, kSmemLimit);
  if (ctas == 0) return SATK_ECUDA;
  // A token's tiles in pieces: one a CTA where there are fewer tokens than CTAs,
  // else as long as six units a CTA even out their lengths or a piece is short.
  m.tiles = (m.a.k + kRows - 1) / kRows;
  m.pieces = 1;
  while (m.pieces < m.tiles && (static_cast<int64_t>(m.a.T) * m.pieces < ctas ||
                                (static_cast<int64_t>(m.a.T) * m.pieces < 6 * ctas &&
                                 m.tiles / (m.pieces * 2) >= kUnitTiles)))
    m.pieces *= 2;
  if (m.pieces > m.tiles) m.pieces = m.tiles;
  m.per = (m.tiles + m.pieces - 1) / m.pieces;
  m.pieces = (m.tiles + m.per - 1) / m.per;
  const int64_t units = static_cast<int64_t>(m.a.T) * m.pieces;
  const int grid = static_cast<int>(units < ctas ? units : ctas);
  m.step_t = grid / m.pieces;
  m.step_piece = grid % m.pieces;
  kernel<<<grid, kThreads, smem, stream>>>(m);
  return launch_status();
}

}  // namespace

// Widths in steps of 16, rows of 16 bytes, counters that stay in 32 bits.
bool latent_weights_mma_fits(const WeightsArgs &a) {
  WeightsMma m;
  int smem;
  return a.D % 16 == 0 && a.cache_rows > 0 && a.T < INT32_MAX - 4096 && a.k < INT32_MAX - 4096 && rows_of_16_bytes(a.q, a.T, a.ld_q_t, a.H, a.ld_q_h) &&
         rows_of_16_bytes(a.cache, a.cache_rows, a.ld_cache, 1, 0) && plan(a, m, smem);
}

int latent_weights_mma(const WeightsArgs &a, int dtype, cudaStream_t stream) {
  WeightsMma m;
  int smem;
  m.a = a;
  if (!plan(a, m, smem)) return SATK_EUNSUPPORTED;
  const bool bf16 = dtype == SATK_BF16;
  if (!tensor_map_16bit(&m.q, bf16, a.q, a.D, a.H, a.H == 1 ? 1024 : a.ld_q_h, m.heads, a.T,
                        a.T == 1 ? static_cast<int64_t>(a.H == 1 ? 1024 : a.ld_q_h) * a.H : a.ld_q_t))
    return SATK_ECUDA;
  // (an entry names a row below 2^31; a map has 2^32 at most)
  const int64_t rows = a.cache_rows > INT32_MAX ? INT32_MAX + 1ll : a.cache_rows;
  if (!tensor_map_16bit(&m.rows, bf16, a.cache, a.D, rows, rows == 1 ? 1024 : a.ld_cache, 1))
    return SATK_ECUDA;
  if (m.slots >= kGroups * kDepth)
    return bf16 ? launch<__nv_bfloat16, kDepth>(m, smem, stream) : launch<__half, kDepth>(m, smem, stream);
  return bf16 ? launch<__nv_bfloat16, 0>(m, smem, stream) : launch<__half, 0>(m, smem, stream);
}

}  // namespace satk
