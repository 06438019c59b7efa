// abi.cu -- status strings, the short-name aliases of the C ABI, and the
// host helpers that keep state (the resident-CTA cache).
#include <cuda.h>
#include <mutex>
#include <unordered_map>

#include "satk_device.cuh"
#include "satk_host.hpp"

namespace satk {

int64_t resident_ctas(const void *kernel, int block, size_t smem) {
  static std::mutex mu;
  static std::unordered_map<const void *, int64_t> cache[64];  // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  {
    std::lock_guard<std::mutex> g(mu);
    auto it = cache[dev].find(kernel);
    if (it != cache[dev].end()) return it->second;
  }
  int sms = 0, per_sm = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem) != cudaSuccess)
    return 0;
  const int64_t n = static_cast<int64_t>(sms) * (per_sm < 1 ? 1 : per_sm);
  std::lock_guard<std::mutex> g(mu);
  cache[dev][kernel] = n;
  return n;
}

bool tensor_map_16bit(void *map, bool bf16, const void *base, int64_t cols, int64_t rows,
                      int64_t ld_rows, int box_rows, int64_t outer, int64_t ld_outer,
                      int box_outer) {
  // The driver's function is looked up through the runtime, so the library
  // needs no link to libcuda; the result is the same for the whole process.
  static const auto encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld_rows) * 2,
                                 static_cast<cuuint64_t>(ld_outer) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows),
                             static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t step[3] = {1, 1, 1};
  const auto make = [&] {
    return encode(static_cast<CUtensorMap *>(map),
                  bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  outer > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (make()) return true;
  // A host thread without a CUDA context (this may be its first call: the
  // runtime gives it one when it launches) is refused by the driver's function.
  // Setting the current device makes its context current.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && make();
}

}  // namespace satk

#ifdef SATK_DEBUG
__device__ unsigned int satk::satk_debug_word;
#endif

extern "C" uint32_t satk_debug_flags(int clear) {
#ifdef SATK_DEBUG
  unsigned int h = 0u;
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpyFromSymbol(&h, satk::satk_debug_word, sizeof h) != cudaSuccess)
    return 0xffffffffu;
  if (clear) {
    const unsigned int z = (clear & 2) != 0 ? satk::kDbgStall : 0u;
    if (cudaMemcpyToSymbol(satk::satk_debug_word, &z, sizeof z) != cudaSuccess) return 0xffffffffu;
  }
  return h;
#else
  (void)clear;
  return 0u;
#endif
}

extern "C" const char *satk_status_string(int rc) {
  switch (rc) {
    case SATK_OK:
      return "ok";
    case SATK_EINVAL:
      return "invalid argument (pointer, size, stride or alignment)";
    case SATK_EUNSUPPORTED:
      return "valid but outside the instantiated range";
    case SATK_ECUDA:
      return "CUDA launch failed";
    default:
      return "unknown status";
  }
}

extern "C" int topk_rows(const void *logits, int dtype, int64_t rows, int64_t cols,
                         int64_t ld_logits, const int32_t *row_ends, int32_t k, int32_t *out,
                         int64_t ld_out, satk_stream_t stream) {
  return satk_topk_rows(logits, dtype, rows, cols, ld_logits, row_ends, k, out, ld_out, stream);
}

extern "C" int topk_rows_sorted(const void *logits, int dtype, int64_t rows, int64_t cols,
                                int64_t ld_logits, const int32_t *row_ends, int32_t k,
                                int32_t *out, int64_t ld_out, satk_stream_t stream) {
  return satk_topk_rows_sorted(logits, dtype, rows, cols, ld_logits, row_ends, k, out, ld_out,
                               stream);
}

extern "C" int dcp_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S, int64_t ld_logits,
                        const int32_t *local_idx, int64_t ld_idx, int32_t n,
                        const int32_t *row_ends, int32_t *packed, satk_stream_t stream) {
  return satk_dcp_pack(logits_bf16, rows, S, ld_logits, local_idx, ld_idx, n, row_ends, packed,
                       stream);
}

extern "C" int dcp_merge_select(const void *cand, int format, int32_t W, int64_t T, int32_t n,
                                int32_t k, int32_t *ids_out, int64_t ld_out, int32_t *sat_word,
                                int32_t *status, satk_stream_t stream) {
  return satk_dcp_merge_select(cand, format, W, T, n, k, ids_out, ld_out, sat_word, status,
                               stream);
}

extern "C" int dcp_rescue_select(const int32_t *packed, int32_t W, int64_t T, int32_t n,
                                 int32_t k, const uint16_t *logits_bf16, int64_t S,
                                 int64_t ld_logits, const int32_t *row_ends,
                                 const int32_t *sat_word, int32_t *recv, int32_t *ids_out,
                                 int64_t ld_out, int32_t *status, satk_stream_t stream) {
  return satk_dcp_rescue_select(packed, W, T, n, k, logits_bf16, S, ld_logits, row_ends,
                                sat_word, recv, ids_out, ld_out, status, stream);
}

extern "C" int dcp_topk_pack(const uint16_t *logits_bf16, int64_t rows, int64_t S,
                             int64_t ld_logits, const int32_t *row_ends, int32_t n,
                             int32_t *packed, satk_stream_t stream) {
  return satk_dcp_topk_pack(logits_bf16, rows, S, ld_logits, row_ends, n, packed, stream);
}
