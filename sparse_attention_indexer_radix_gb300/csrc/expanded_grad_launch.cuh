// expanded_grad_launch.cuh -- the backward pass of the expanded attention on the
// tensor cores: one launch for both kernels, so that the CTAs of one fill the SMs
// that the other leaves idle at its end.  Those of the queries come first: each takes
// about as long as the longest of the keys', whose last ones, with few tokens, come
// last.  FEW: see kFewTokens.
#pragma once

#include "expanded_grad_keys.cuh"
#include "expanded_grad_tokens.cuh"

namespace satk {

struct GradMma {
  ExpandedGradArgs a;
  GradShape s;
  GradMaps maps;
  grad_keys::Plan keys;
  grad_tokens::Plan tokens;
  unsigned token_blocks, key_blocks;
};

template <class E, bool FEW>
__global__ void __launch_bounds__(kGradThreads, 1) expanded_grad_mma_kernel(const __grid_constant__ GradMma m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  wait_for_previous_kernel();  // the tokens' statistics
  let_next_kernel_start();
  if (blockIdx.x < m.token_blocks)
    grad_tokens::run<E, FEW>(m.a, m.s, m.tokens, m.maps, smem, blockIdx.x, m.token_blocks);
  else
    grad_keys::run<E, FEW>(m.a, m.s, m.keys, m.maps, smem, blockIdx.x - m.token_blocks, m.key_blocks);
}

template <class E, bool FEW>
int launch_grad_mma(const GradMma &m, int smem, cudaStream_t stream) {
  if (!allow_smem(expanded_grad_mma_kernel<E, FEW>, smem, kSmemLimit)) return SATK_ECUDA;
  return launch_early(expanded_grad_mma_kernel<E, FEW>, m.token_blocks + m.key_blocks, kGradThreads, smem, stream, m);
}

// Compiled in a file of its own, beside the other.
int launch_grad_few(const GradMma &m, bool bf16, int smem, cudaStream_t stream);

}  // namespace satk
