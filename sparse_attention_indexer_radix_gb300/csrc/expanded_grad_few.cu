// expanded_grad_few.cu -- the backward pass of the expanded attention on the tensor
// cores for calls of few tokens a request.
#include "expanded_grad_launch.cuh"

namespace satk {

int launch_grad_few(const GradMma &m, bool bf16, int smem, cudaStream_t stream) {
  return bf16 ? launch_grad_mma<__nv_bfloat16, true>(m, smem, stream)
              : launch_grad_mma<__half, true>(m, smem, stream);
}

}  // namespace satk
