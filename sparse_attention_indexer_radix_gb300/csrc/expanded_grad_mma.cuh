// expanded_grad_mma.cuh -- what the two tensor-core kernels of the expanded
// attention's backward pass share.
#pragma once

#include <cuda.h>
#include <type_traits>

#include "expanded_grad.cuh"
#include "satk_tcgen05.cuh"

namespace satk {

constexpr int kGradThreads = 384;  // warps 0-7 elementwise, 8 MMAs, 9 loads, 10 and 11 rows
constexpr int kTile = 128;         // rows of the tile that a CTA owns
constexpr int kMaxPanels = 5;      // 64-column panels of a query or key (dn, then the tail)

// The inputs, all read in boxes of 64 columns x 64 rows of a head.
constexpr int kBoxRows = 64;
struct GradMaps {
  CUtensorMap q, dout, k, tail, v;
};

// Widths in panels, and where a CTA's work lies.
struct GradShape {
  int nope_panels, panels, v_panels;
  int one_product;  // one product gives all of the query's or key's columns (no gap before the tail)
  int full;         // no panel has fewer than 64 columns
  int gap;          // columns of tensor memory that the nope part's last panel lacks
  int vec_k, vec_v, vec_q;  // 16-byte aligned gradient rows
};

// The request whose tiles of kTile rows have this slot, by a whole warp: the last
// one whose first slot, starts[r] / kTile + r, is at or before it.
__device__ __forceinline__ int request_of_slot(const int32_t *starts, int R, int n, int slot) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, r = lo + lane * step;
    const bool before = r < hi && (lane == 0 || span_of(starts, r, n).begin / kTile + r <= slot);
    const int count = __popc(__ballot_sync(~0u, before));
    lo += (count - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// One row of a tile in `panels` 128-byte-swizzled panels `stride` bytes apart:
// whether a value is not finite, and zeros in its place.  A row's chunks are read
// from another one on for every lane, clear of bank conflicts.
template <class E>
__device__ __forceinline__ bool row_is_odd(const unsigned char *tile, int row, int panels, int stride) {
  typename Elem<E>::T2 sum = Elem<E>::from2(0.f, 0.f), zero = sum;
  for (int p = 0; p < panels; ++p) {
    const unsigned char *at = tile + p * stride + row * 128;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      Pack8<E> c;
      c.u = *reinterpret_cast<const uint4 *>(at + ((x ^ (row & 7)) << 4));
#pragma unroll
      for (int z = 0; z < 4; ++z) sum = __hfma2(c.h[z], zero, sum);  // NaN: not finite
    }
  }
  const float2 f = Elem<E>::to2(sum);
  return !(f.x == 0.f && f.y == 0.f);
}
__device__ __forceinline__ void clear_row(unsigned char *tile, int row, int panels, int stride) {
  for (int p = 0; p < panels; ++p)
#pragma unroll
    for (int x = 0; x < 8; ++x)
      *reinterpret_cast<uint4 *>(tile + p * stride + row * 128 + (x << 4)) = make_uint4(0, 0, 0, 0);
}

// Up to 64 columns (a multiple of 16; of float: 32) of a warp's 32 rows from tensor
// memory to the first `rows` of them at `to` (`rows` may be more than the warp has: what
// is left of the tile).  They are turned through the warp's own 4 KB of shared memory:
// with rows of 16-byte chunks a store then covers whole lines of four rows and not 16
// bytes of each of 32.  `some`: there is something in tensor memory.
template <class O>
__device__ __forceinline__ void store_rows(unsigned char *turn, uint32_t tmem, int cols, bool some, float scale,
                                           O *to, int64_t ld, int rows, bool vec) {
  constexpr int kChunk = 16 / sizeof(O);  // values
  const int lane = threadIdx.x & 31;
  for (int c = 0; c < cols; c += 16) {
    uint32_t x[16] = {};
    if (some) {
      tmem_ld16(x, tmem + c);
      tmem_wait_ld();
    }
    uint4 chunk[sizeof(O)];
    if constexpr (sizeof(O) == 4) {
#pragma unroll
      for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * scale);
#pragma unroll
      for (int y = 0; y < 4; ++y) chunk[y] = make_uint4(x[4 * y], x[4 * y + 1], x[4 * y + 2], x[4 * y + 3]);
    } else {
      Pack8<O> p[2];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        p[y >> 2].h[y & 3] = Elem<O>::from2(__uint_as_float(x[2 * y]) * scale, __uint_as_float(x[2 * y + 1]) * scale);
      chunk[0] = p[0].u, chunk[1] = p[1].u;
    }
#pragma unroll
    for (int y = 0; y < static_cast<int>(sizeof(O)); ++y)
      *reinterpret_cast<uint4 *>(turn + lane * 128 + (((c / kChunk + y) ^ (lane & 7)) << 4)) = chunk[y];
  }
  __syncwarp();
  if (vec) {
    const int ch = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (r < rows && ch * kChunk < cols)
        *reinterpret_cast<uint4 *>(to + r * ld + ch * kChunk) =
            *reinterpret_cast<const uint4 *>(turn + r * 128 + ((ch ^ (r & 7)) << 4));
    }
  } else {
    const int n = min(rows, 32) * cols;
    for (int i = lane; i < n; i += 32) {
      const int r = i / cols, c = i - r * cols;
      to[r * ld + c] = *reinterpret_cast<const O *>(turn + r * 128 + (((c / kChunk) ^ (r & 7)) << 4) +
                                                    (c % kChunk) * sizeof(O));
    }
  }
  __syncwarp();
}

// The same rows and columns after a wait that was given up: NaN, straight to memory (a
// copy may still be on its way to any shared memory).
template <class O>
__device__ __forceinline__ void lose_rows(O *to, int64_t ld, int rows, int cols) {
  O nan;
  if constexpr (sizeof(O) == 4) nan = NAN; else nan = Elem<O>::from(NAN);
  const int n = min(rows, 32) * cols;
  for (int i = threadIdx.x & 31; i < n; i += 32) to[i / cols * ld + i % cols] = nan;
}

// The rows of no request, of one head: zeros by whole warps.
template <class F>
__device__ __forceinline__ void rows_outside(const int32_t *starts, int R, int n, F zero) {
  const int b = R > 0 ? min(max(starts[0], 0), n) : n;
  const int e = R > 0 ? min(max(starts[R], b), n) : n;
  const int warp = threadIdx.x >> 5, warps = kGradThreads / 32;
  for (int64_t i = warp; i < b; i += warps) zero(i);
  for (int64_t i = e + warp; i < n; i += warps) zero(i);
}

// P and dS are operands of 16 bits: each is off by up to half a step of itself.  Over
// many tokens these errors average out, the result's own rounding is as large; over
// two to eight tokens they do not always (an error of up to 1.8 times that of the
// formula with 32-bit P and dS where 1.4 is usual, in 10 of 240 gradients).  Requests of
// one tile of tokens take a second operand that holds what the rounding left (none is
// above 1.5 then): 8 requests of 8 tokens behind 2000 keys, 16 heads, take 199 us (one
// operand: 182).  The request alone decides, so its bits do not depend on what else is
// in the call; requests of many tokens pay for code that they do not run (five prompts of
// up to 391 tokens 46 us for 44, packed prompts 122 for 120, a chunk 624 for 622).
constexpr int kFewTokens = 64;

// Two values rounded to 16 bits, and what the rounding left of them likewise: as two
// operands they stand for some 16 bits of fraction.
template <class E>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  union {
    typename Elem<E>::T2 h;
    uint32_t u;
  } pk;
  pk.h = Elem<E>::from2(x, y);
  return pk.u;
}
template <class E>
__device__ __forceinline__ uint32_t pack16_rest(float x, float y, uint32_t rounded) {
  union {
    typename Elem<E>::T2 h;
    uint32_t u;
  } pk;
  pk.u = rounded;
  const float2 r = Elem<E>::to2(pk.h);
  // (nothing is left of what is not finite, or is too large for the type)
  const float a = x - r.x, b = y - r.y;
  return pack16<E>(fabsf(r.x) < INFINITY ? a : 0.f, fabsf(r.y) < INFINITY ? b : 0.f);
}

// Which steps of 16 columns there are, four bits a panel.
__device__ __forceinline__ uint32_t panel_steps(int panels, int nope_panels, int dn, int dr) {
  uint32_t steps = 0;
  for (int p = 0; p < panels; ++p) {
    const int cols = p >= nope_panels ? dr : p == nope_panels - 1 ? dn - p * 64 : 64;
    steps |= ((1u << (cols >> 4)) - 1) << (4 * p);
  }
  return steps;
}

// A product over columns, both operands K-major in PANELS panels: A in shared memory
// (panels A_PANEL bytes apart) or, INSIDE, in tensor memory without gaps (`gap`: what
// the last panel but one lacks there).  FULL: every panel has all its steps.
template <bool INSIDE, int PANELS, bool FULL, int A_PANEL, int B_PANEL>
__device__ __forceinline__ void product_over_columns(uint32_t d, uint32_t a, uint32_t b, uint32_t desc,
                                                     uint32_t steps, uint32_t gap) {
#pragma unroll
  for (int p = 0; p < PANELS; ++p) {
    uint32_t at = a + p * (INSIDE ? 32 : A_PANEL >> 4);
    if (INSIDE && !FULL && p == PANELS - 1) at -= gap;
    const uint32_t bt = b + p * (B_PANEL >> 4);
    if (INSIDE) mma_ts_low(d, at, bt, desc, p > 0); else mma_ss_low(d, at, bt, desc, p > 0);
#pragma unroll
    for (int x = 1; x < 4; ++x) {
      const bool on = FULL || (steps >> (4 * p + x) & 1u) != 0;
      if (INSIDE) mma_ts_low_if(on, d, at + 8 * x, bt + 2 * x, desc);
      else mma_ss_low_if(on, d, at + 2 * x, bt + 2 * x, desc);
    }
  }
}

template <int N>
using Const = std::integral_constant<int, N>;

// issue(panels, panels of the values, whether all are full) with constants.
template <class F>
__device__ __forceinline__ void with_shape(int panels, int v_panels, bool full, F issue) {
  auto values = [&](auto np) {
    if (full) {
      if (v_panels == 1) issue(np, Const<1>(), Const<1>()); else issue(np, Const<2>(), Const<1>());
    } else {
      if (v_panels == 1) issue(np, Const<1>(), Const<0>()); else issue(np, Const<2>(), Const<0>());
    }
  };
  if (panels == 1) values(Const<1>());
  else if (panels == 2) values(Const<2>());
  else if (panels == 3) values(Const<3>());
  else if (panels == 4) values(Const<4>());
  else values(Const<5>());
}

}  // namespace satk
