// expanded_grad_mma.cu -- the backward pass of the expanded attention on the tensor
// cores: what it takes, its shared memory and tensor maps, its launch.
//
// One launch for both kernels, so that the CTAs of one fill the SMs that the other
// leaves idle at its end.  Those of the queries come first: each takes about as long as
// the longest of the keys', whose last ones, with few tokens, come last.
#include "expanded_grad_keys.cuh"
#include "expanded_grad_tokens.cuh"

namespace satk {
namespace {

struct GradMma {
  ExpandedGradArgs a;
  GradShape s;
  GradMaps maps;
  grad_keys::Plan keys;
  grad_tokens::Plan tokens;
  unsigned token_blocks, key_blocks;
};

template <class E>
__global__ void __launch_bounds__(kGradThreads, 1) expanded_grad_mma_kernel(const __grid_constant__ GradMma m) {
  extern __shared__ __align__(1024) unsigned char smem[];
  wait_for_previous_kernel();  // the tokens' statistics
  let_next_kernel_start();
  if (blockIdx.x < m.token_blocks)
    grad_tokens::run<E>(m.a, m.s, m.tokens, m.maps, smem, blockIdx.x, m.token_blocks);
  else
    grad_keys::run<E>(m.a, m.s, m.keys, m.maps, smem, blockIdx.x - m.token_blocks, m.key_blocks);
}

template <class E>
int launch(const GradMma &m, int smem, cudaStream_t stream) {
  if (!allow_smem(expanded_grad_mma_kernel<E>, smem, kSmemLimit)) return SATK_ECUDA;
  return launch_early(expanded_grad_mma_kernel<E>, m.token_blocks + m.key_blocks, kGradThreads, smem, stream, m);
}

GradShape shape_of(const ExpandedGradArgs &a) {
  const ExpandedArgs &f = a.f;
  GradShape s;
  s.nope_panels = (f.dn + 63) / 64;
  s.panels = s.nope_panels + (f.dr > 0 ? 1 : 0);
  s.v_panels = (f.dv + 63) / 64;
  s.one_product = f.dr == 0 || f.dn % 64 == 0;
  s.full = f.dn % 64 == 0 && f.dr % 64 == 0 && f.dv % 64 == 0;
  s.gap = f.dr > 0 ? (s.nope_panels * 64 - f.dn) / 2 : 0;
  s.vec_k = rows_of_16_bytes(a.dk, f.S, a.ld_dk_s, f.H, a.ld_dk_h);
  s.vec_v = rows_of_16_bytes(a.dv, f.S, a.ld_dv_s, f.H, a.ld_dv_h);
  s.vec_q = rows_of_16_bytes(a.dq, f.T, a.ld_dq_t, f.H, a.ld_dq_h);
  return s;
}

bool maps_of(const ExpandedGradArgs &a, bool bf16, GradMaps &m) {
  const ExpandedArgs &f = a.f;
  // [n, H, cols]; strides of dimensions of one are free, any multiple of 16 bytes.
  const auto heads = [&](CUtensorMap *to, const void *p, int cols, int64_t n, int64_t ld, int64_t ld_h) {
    return tensor_map_16bit(to, bf16, p, cols, f.H, f.H == 1 ? 1024 : ld_h, 1, n, n == 1 ? 1024 : ld, kBoxRows);
  };
  return heads(&m.q, f.q, f.dn + f.dr, f.T, f.ld_q_t, f.ld_q_h) &&
         heads(&m.dout, a.dout, f.dv, f.T, a.ld_do_t, a.ld_do_h) &&
         heads(&m.k, f.k, f.dn, f.S, f.ld_k_s, f.ld_k_h) && heads(&m.v, f.v, f.dv, f.S, f.ld_v_s, f.ld_v_h) &&
         (f.dr == 0 ||
          tensor_map_16bit(&m.tail, bf16, f.tail, f.dr, f.S, f.S == 1 ? 1024 : f.ld_tail, kBoxRows));
}

}  // namespace

// Widths in steps of 16, rows of 16 bytes, something to see.
bool expanded_grad_mma_fits(const ExpandedGradArgs &a) {
  const ExpandedArgs &f = a.f;
  const GradShape s = shape_of(a);
  GradMma m;
  int smem;
  return f.T > 0 && f.S > 0 && f.R > 0 && f.dn % 16 == 0 && f.dr % 16 == 0 && f.dv % 16 == 0 &&
         f.dr <= 64 && s.panels <= kMaxPanels && rows_of_16_bytes(f.q, f.T, f.ld_q_t, f.H, f.ld_q_h) &&
         rows_of_16_bytes(a.dout, f.T, a.ld_do_t, f.H, a.ld_do_h) &&
         rows_of_16_bytes(f.k, f.S, f.ld_k_s, f.H, f.ld_k_h) &&
         rows_of_16_bytes(f.v, f.S, f.ld_v_s, f.H, f.ld_v_h) &&
         (f.dr == 0 || rows_of_16_bytes(f.tail, f.S, f.ld_tail, 1, 0)) &&
         grad_keys::plan(a, s, m.keys, smem) && grad_tokens::plan(a, s, m.tokens, smem);
}

int expanded_grad_mma(const ExpandedGradArgs &a, int dtype, cudaStream_t stream) {
  GradMma m;
  m.a = a;
  m.s = shape_of(a);
  const bool bf16 = dtype == SATK_BF16;
  int keys_smem, tokens_smem;
  if (!grad_keys::plan(a, m.s, m.keys, keys_smem) || !grad_tokens::plan(a, m.s, m.tokens, tokens_smem))
    return SATK_EUNSUPPORTED;
  if (!maps_of(a, bf16, m.maps)) return SATK_ECUDA;
  // (one more CTA a head for the rows of no request)
  const int64_t tokens = (tile_slots(a.f.T, a.f.R, kTile) + 1) * a.f.H;
  const int64_t keys = (tile_slots(a.f.S, a.f.R, kTile) + 1) * a.f.H;
  if (tokens + keys > INT32_MAX) return SATK_EUNSUPPORTED;
  m.token_blocks = static_cast<unsigned>(tokens);
  m.key_blocks = static_cast<unsigned>(keys);
  const int smem = keys_smem > tokens_smem ? keys_smem : tokens_smem;
  return bf16 ? launch<__nv_bfloat16>(m, smem, stream) : launch<__half>(m, smem, stream);
}

}  // namespace satk
