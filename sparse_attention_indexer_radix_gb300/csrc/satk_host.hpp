// satk_host.hpp -- host-side helpers shared by the entry points of
// libsatk.so: argument checks, launch-status mapping, stream cast.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "satk.h"

namespace satk {

inline cudaStream_t as_stream(satk_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// log2 of a power of two, else -1.
inline int log2_or(int v) {
  if (v <= 0 || (v & (v - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Maps the result of the launches just issued to an SATK return code.
inline int launch_status() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SATK_OK : SATK_ECUDA;
}

// Lets a launch of `kernel` take `bytes` of dynamic shared memory.  `most` is
// the largest size that any call of this kernel takes (0: it always takes
// `bytes`).  The limit set is `most` every time, never a call's own size: it is
// the kernel's for the whole process, and another thread may be about to launch
// with more.
template <class K>
inline bool allow_smem(K kernel, size_t bytes, size_t most = 0) {
  // A block has 48 KB without asking, for what the kernel declares statically too.
  if (bytes <= 32 * 1024) return true;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(most > bytes ? most : bytes)) == cudaSuccess;
}

// All the shared memory that a block may have.
constexpr int kSmemLimit = 227 * 1024;

// CTAs of `kernel` (block threads, smem dynamic bytes) the current device
// holds at once: SMs x resident CTAs per SM, computed once per kernel and
// device.  0 on error.
int64_t resident_ctas(const void *kernel, int block, size_t smem);

// The tensor map of 16-bit elements [outer, rows, cols] (strides in elements;
// base and strides multiples of 16 bytes) read in boxes of 64 columns x box_rows
// x box_outer with the 128-byte swizzle; what a box covers outside the tensor
// reads as zeros.  outer = 0: a matrix [rows, cols].  False if the driver
// refuses it.
bool tensor_map_16bit(void *map, bool bf16, const void *base, int64_t cols, int64_t rows,
                      int64_t ld_rows, int box_rows, int64_t outer = 0, int64_t ld_outer = 0,
                      int box_outer = 1);

}  // namespace satk
