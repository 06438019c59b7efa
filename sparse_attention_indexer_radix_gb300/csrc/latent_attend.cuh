// latent_attend.cuh -- arguments of the attention over latent cache rows and
// the key addressing that its kernels share.
#pragma once

#include "latent_common.cuh"

namespace satk {

struct LatentArgs {
  const void *q;
  int T, H, dl, D;  // D = dl + dr
  int64_t ld_q_t, ld_q_h;
  const void *cache;
  int64_t cache_rows, ld_cache;
  // paged keys (rows == nullptr)
  const int32_t *req_id, *block_table;
  int64_t table_rows, ld_table;
  int max_keys;  // max_blocks * block_size, the table's reach in local tokens
  int block_size, b_shift;
  int64_t stride_rows;
  const int32_t *row_ends, *tree;
  int tree_words;
  // selected keys
  const int32_t *rows, *counts;
  int64_t ld_rows;
  int k;
  float scale_log2;  // scale * log2(e): scores and statistics are kept in log2
  void *out;
  int64_t ld_out_t, ld_out_h;
  float *lse;
  int32_t *status;
};

// Keys [0, end) that token t sees unconditionally (paged: its causal end;
// selected: its entries).  0 and a status bit for a request outside the table.
__device__ __forceinline__ int token_end(const LatentArgs &a, int t) {
  if (a.rows != nullptr) return a.counts == nullptr ? a.k : min(max(a.counts[t], 0), a.k);
  const int r = a.req_id[t];
  if (r < 0 || r >= a.table_rows) {
    if (a.status != nullptr) atomicOr(a.status, SATK_STATUS_BAD_REQUEST);
    return 0;
  }
  return min(max(a.row_ends[t], 0), a.max_keys);
}

// Does token t see its request's key end + b of the drafted tree?
__device__ __forceinline__ bool tree_bit(const LatentArgs &a, int t, int b) {
  if (b < 0 || b >= a.tree_words * 32) return false;
  return (a.tree[static_cast<int64_t>(t) * a.tree_words + (b >> 5)] >> (b & 31)) & 1;
}

// One past the last key that token t may see, its tree's bits included.
__device__ __forceinline__ int token_extent(const LatentArgs &a, int t, int end) {
  if (a.rows != nullptr || a.tree == nullptr) return end;
  const int r = a.req_id[t];
  if (r < 0 || r >= a.table_rows) return 0;
  const int first = max(a.row_ends[t], 0);
  for (int w = a.tree_words - 1; w >= 0; --w) {
    const unsigned bits = a.tree[static_cast<int64_t>(t) * a.tree_words + w];
    if (bits != 0) {
      const int64_t last = static_cast<int64_t>(first) + w * 32 + 32 - __clz(bits);
      return max(end, static_cast<int>(min(last, static_cast<int64_t>(a.max_keys))));
    }
  }
  return end;
}

// The load behind key j of token t: its row, or its block. The row itself, or -1
// (a skipped entry, or a row outside the cache, which raises its status bit),
// comes from it in a second step, so that the load can be in flight meanwhile.
__device__ __forceinline__ int key_entry(const LatentArgs &a, int t, int r, int j) {
  if (a.rows != nullptr) return a.rows[t * a.ld_rows + j];
  return a.block_table[r * a.ld_table + (a.b_shift >= 0 ? j >> a.b_shift : j / a.block_size)];
}
__device__ __forceinline__ int64_t entry_row(const LatentArgs &a, int entry, int j) {
  int64_t row = entry;
  if (a.rows != nullptr) {
    if (row < 0) return -1;
  } else {
    row = row * a.stride_rows +
          (a.b_shift >= 0 ? j & ((1 << a.b_shift) - 1) : j % a.block_size);
  }
  if (row < 0 || row >= a.cache_rows) {
    if (a.status != nullptr) atomicOr(a.status, SATK_STATUS_BAD_ROW);
    return -1;
  }
  return row;
}
__device__ __forceinline__ int64_t key_row(const LatentArgs &a, int t, int r, int j) {
  return entry_row(a, key_entry(a, t, r, j), j);
}

// The general kernel: any widths, strides and alignment (latent_attend_warp.cu).
int latent_attend_warp(const LatentArgs &a, int dtype, cudaStream_t stream);

// The tensor-core kernel (latent_attend_mma.cu): whether it takes this call, its
// workspace, and the call; tokens_per_request is the host's estimate.
bool latent_attend_mma_fits(const LatentArgs &a);
size_t latent_attend_mma_workspace(int H, int dl);
int latent_attend_mma(const LatentArgs &a, int dtype, int tokens_per_request, void *workspace,
                      cudaStream_t stream);

}  // namespace satk
