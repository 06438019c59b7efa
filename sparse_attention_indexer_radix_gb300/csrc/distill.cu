// distill.cu -- the distillation loss of a row of scores against a teacher's
// entries, and the gradient of the scores.
//
// loss: a cluster of 1 to 8 CTAs takes a row.  Every thread keeps a running
// maximum and the sum of exponentials of its share of the visible columns (one
// pass); the CTA, then the cluster, joins them, and the row's first CTA weighs the
// entries, whose scores it gathered before the pass.  Differences to the maximum
// are taken before they are scaled, so scores of any size and offset keep their
// digits.  Over the entries alone nothing but the gather remains.
//
// grad: a CTA takes up to 32768 columns of a row.  It writes the student's part of
// every column as a stream, then the few entries' columns again, whole, from
// the scores it read before (so the gradient may take the scores' place).  A bit
// a column finds entries that share one: a warp sums those, in the entries'
// order, so no result depends on the order in which threads arrive.
//
// Both are bound by memory: one exponential an element, 2 or 4 bytes read (and
// written).  4096 causal rows of up to 51200 fp32 columns: loss 129 us, 6.4 TB/s; 2048
// rows of 102400 bf16 columns: gradient 137 us, 6.1 TB/s; 512 entries of 4096 rows:
// loss 31 us, most of it 64 bytes of DRAM an entry.
#include <algorithm>
#include <cooperative_groups.h>

#include "distill.cuh"

namespace cg = cooperative_groups;

namespace satk {
namespace {

constexpr int kChunk = 32768;       // columns of a gradient CTA at most
constexpr int kLeastChunk = 4096;   // columns worth a CTA of their own
constexpr int kMostCluster = 8;
constexpr int kUnroll = 4;

__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// Running maximum and sum of exponentials (raw scores; c scales to log2).
struct Running {
  float m = -INFINITY;
  float2 l = make_float2(0.f, 0.f);
  __device__ __forceinline__ void raise(float mx, float c) {
    if (mx > m) {
      const float f = exp2_fast((m - mx) * c);
      l.x *= f;
      l.y *= f;
      m = mx;
    }
  }
};

template <class E, int N>
__device__ __forceinline__ void take(Running &r, const uint4 (&u)[N], float c) {
  constexpr int kP = Vec16<E>::kN / 2;
  float2 f[N * kP];
#pragma unroll
  for (int i = 0; i < N; ++i) Vec16<E>::to(u[i], f + i * kP);
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < N * kP; ++i) mx = fmaxf(mx, fmaxf(f[i].x, f[i].y));
  r.raise(mx, c);
  const float ref = finite_or_0(r.m);
  const float2 less = make_float2(-ref, -ref), c2 = make_float2(c, c);
#pragma unroll
  for (int i = 0; i < N * kP; ++i) {
    float2 x = __fmul2_rn(__fadd2_rn(f[i], less), c2);
    x.x = exp2_fast(x.x);
    x.y = exp2_fast(x.y);
    r.l = __fadd2_rn(r.l, x);
  }
}

// Columns [b, e) of a row into a thread's running sum.
template <class E>
__device__ __forceinline__ void scan(Running &r, const E *row, int b, int e, float c) {
  constexpr int kN = Vec16<E>::kN;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row + b) & 15) / sizeof(E));
  const int first = min(e, b + (off == 0 ? 0 : kN - off));
  auto one = [&](int v) {
    const float x = Elem<E>::to(row[v]);
    r.raise(x, c);
    r.l.x += exp2_fast((x - finite_or_0(r.m)) * c);
  };
  if (static_cast<int>(threadIdx.x) < first - b) one(b + threadIdx.x);
  const int n = (e - first) / kN;
  const uint4 *at = reinterpret_cast<const uint4 *>(row + first);
  const uint4 none = [] {
    float2 f[4];
    for (int i = 0; i < 4; ++i) f[i] = make_float2(-INFINITY, -INFINITY);
    return Vec16<E>::from(f);
  }();
  for (int i = threadIdx.x; i < n; i += kUnroll * kDistillThreads) {
    uint4 u[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int x = i + j * kDistillThreads;
      u[j] = x < n ? ldg_stream(at + x) : none;
    }
    take<E, kUnroll>(r, u, c);
  }
  const int last = first + n * kN;
  if (static_cast<int>(threadIdx.x) < e - last) one(last + threadIdx.x);
}

// The two halves of a cluster barrier, of all threads of all its CTAs.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <class E, int PER, bool LISTED>
__global__ void __launch_bounds__(kDistillThreads) distill_loss_kernel(DistillArgs a) {
  __shared__ float2 part[kDistillThreads / 32];
  __shared__ float2 joined[kMostCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = static_cast<int>(cluster.num_blocks());
  const int rank = static_cast<int>(cluster.block_rank());
  // (said here, waited for behind the pass: the first CTA's shared memory may be
  // written once it has started)
  if (ctas > 1) cluster_arrive();
  const int64_t t = blockIdx.x / ctas;
  const E *row = static_cast<const E *>(a.logits) + t * a.ld;
  const int end = row_end(a, t);
  Entries<PER> in;
  float s[PER];
  if (rank == 0) {
    in.load(a, t, end);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = in.id[i] >= 0 ? Elem<E>::to(row[in.id[i]]) : -INFINITY;
  }
  Running r;
  if (LISTED) {
#pragma unroll
    for (int i = 0; i < PER; ++i) r.m = fmaxf(r.m, s[i]);
  } else {
    const int64_t per = (end / ctas + 8) & ~7;
    const int b = static_cast<int>(min(static_cast<int64_t>(end), rank * per));
    scan(r, row, b, static_cast<int>(min(static_cast<int64_t>(end), b + per)), a.c);
  }
  // Maxima of the student's scores and, in the row's first CTA, the teacher's.
  float top = -INFINITY;
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, in.x[i]);
  }
  const float2 most = block_reduce2<true>(make_float2(r.m, top), part);
  float ref = finite_or_0(most.x);
  const float x_ref = finite_or_0(most.y);
  const float unit = a.kind == SATK_TEACHER_WEIGHTS ? list_scale(most.y) : 1.f;
  if (LISTED) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (in.id[i] >= 0) r.l.x += exp2_fast((s[i] - ref) * a.c);
  } else {
    r.l.x = (r.l.x + r.l.y) * exp2_fast((r.m - ref) * a.c);
  }
  // The teacher's total, unless its values are shares already.
  float total = 0.f;
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (in.id[i] < 0) continue;
      total += a.kind == SATK_TEACHER_LOGITS ? exp2_fast((in.x[i] - x_ref) * a.c) : in.x[i] * unit;
    }
  }
  float2 sums = block_reduce2<false>(make_float2(r.l.x, total), part);
  float m = most.x;
  if (ctas > 1) {
    cluster_wait();
    if (threadIdx.x == 0) cluster.map_shared_rank(joined, 0)[rank] = make_float2(m, sums.x);
    cluster.sync();
    if (rank != 0) return;
    m = -INFINITY;
    for (int i = 0; i < ctas; ++i) m = fmaxf(m, joined[i].x);
    ref = finite_or_0(m);
    sums.x = 0.f;
    for (int i = 0; i < ctas; ++i) sums.x += joined[i].y * exp2_fast((joined[i].x - ref) * a.c);
  }
  // loss = sum p (log p - (s - m) / tau) + log(sum of exponentials) sum p
  const float log_l = log2f(sums.x) * kLn2;
  float loss = 0.f, mass = 0.f;
  const float scale = a.kind == SATK_TEACHER_PROBS ? 1.f : 1.f / sums.y;
  const float log_total = a.kind == SATK_TEACHER_PROBS ? 0.f : logf(sums.y);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (in.id[i] < 0) continue;
    float w, log_w;
    if (a.kind == SATK_TEACHER_LOGITS) {
      log_w = (in.x[i] - x_ref) * a.inv_tau;
      w = exp2_fast((in.x[i] - x_ref) * a.c);
    } else {
      w = in.x[i] * unit;
      log_w = logf(w);
    }
    if (w == 0.f) continue;
    w *= scale;
    mass += w;
    loss += w * ((log_w - log_total) - (s[i] - ref) * a.inv_tau);
  }
  const float2 all = block_reduce2<false>(make_float2(loss, mass), part);
  if (threadIdx.x == 0) {
    // (a teacher without any mass asks for nothing)
    a.loss[t] = sums.y == 0.f ? 0.f : all.x + all.y * log_l;
    a.lse[t] = m == -INFINITY ? (sums.x == 0.f ? -INFINITY : NAN) : m * a.inv_tau + log_l;
  }
}

// A bit a column: it has an entry, it has several; the columns that have several,
// with their scores.
template <int ENTRIES>
struct Listed {
  float2 part[kDistillThreads / 32];
  uint32_t any[kChunk / 32], several[kChunk / 32];
  int column[ENTRIES / 2];
  float score[ENTRIES / 2];
  int n;
};

// (plain loads: the gradient may take the place of the scores)
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ float min_or_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

template <class E, int PER, bool LISTED>
__global__ void __launch_bounds__(kDistillThreads) distill_grad_kernel(DistillArgs a) {
  constexpr int kN = Vec16<E>::kN;
  constexpr int kLoads = LISTED ? 2 : kUnroll;  // (zeros need no registers, CTAs do)
  __shared__ Listed<PER * kDistillThreads> sm;
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x / a.chunks;
  const int b = static_cast<int>(blockIdx.x % a.chunks) * a.chunk;
  const int e = static_cast<int>(min(a.cols, static_cast<int64_t>(b) + a.chunk));
  const E *row = static_cast<const E *>(a.logits) + t * a.ld;
  E *out = static_cast<E *>(a.grad) + t * a.ld_grad;
  const int end = row_end(a, t);
  const float g = a.dloss[t * a.dloss_step] * a.inv_tau;
  const float less = -a.lse_in[t];
  // The student's share of a score: the difference to lse first, so that only its own
  // size is rounded on the way to log2; at most 1, also where scores are so large that
  // lse has lost the digits behind the point.
  auto share = [&](float s) { return exp2_fast(min_or_nan(fmaf(s, a.inv_tau, less), 0.f) * kLog2e); };
  Entries<PER> in;
  in.load(a, t, end);
  const int words = (e - b + 31) / 32;
  for (int i = tid; i < words; i += kDistillThreads) sm.any[i] = sm.several[i] = 0;
  if (tid == 0) sm.n = 0;

  // The teacher's shares.
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, in.x[i]);
  top = block_reduce2<true>(make_float2(top, 0.f), sm.part).x;
  const float x_ref = finite_or_0(top);
  const float unit = a.kind == SATK_TEACHER_WEIGHTS ? list_scale(top) : 1.f;
  auto weight = [&](float x) {
    return a.kind == SATK_TEACHER_LOGITS ? exp2_fast((x - x_ref) * a.c) : x * unit;
  };
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (in.id[i] >= 0) total += weight(in.x[i]);
  total = block_reduce2<false>(make_float2(total, 0.f), sm.part).x;
  const float norm = a.kind == SATK_TEACHER_PROBS ? 1.f : 1.f / total;
  const float mass = a.kind == SATK_TEACHER_PROBS ? total : total == total ? 1.f : NAN;
  // A row that asks for nothing gets zeros, whatever its scores are.
  const bool asks = total != 0.f && g != 0.f;

  // This chunk's entries: their scores, and which of them write a column.
  float s[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int v = in.id[i];
    s[i] = 0.f;
    if (!asks || v < b || v >= e) {
      in.id[i] = -1;
      continue;
    }
    s[i] = Elem<E>::to(row[v]);
    const uint32_t bit = 1u << ((v - b) & 31);
    if ((atomicOr(&sm.any[(v - b) >> 5], bit) & bit) != 0) {
      atomicOr(&sm.several[(v - b) >> 5], bit);
      in.id[i] = -1;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int v = in.id[i];
    if (v >= 0 && (sm.several[(v - b) >> 5] >> ((v - b) & 31) & 1) != 0) {
      const int at = atomicAdd(&sm.n, 1);
      sm.column[at] = v;
      sm.score[at] = s[i];
      in.id[i] = -1;
    }
  }

  // Every column: the student's part up to the row's end, zeros behind it.
  const float coef = g * mass;
  const int live = LISTED || !asks ? b : min(max(end, b), e);
  auto one = [&](int v) { out[v] = Elem<E>::from(v < live ? share(Elem<E>::to(row[v])) * coef : 0.f); };
  const uintptr_t at_out = reinterpret_cast<uintptr_t>(out + b);
  if (((reinterpret_cast<uintptr_t>(row + b) ^ at_out) & 15) == 0 || live == b) {
    const int off = static_cast<int>((at_out & 15) / sizeof(E));
    const int first = min(e, b + (off == 0 ? 0 : kN - off));
    const int n = (e - first) / kN, last = first + n * kN;
    if (tid < first - b) one(b + tid);
    if (tid < e - last) one(last + tid);
    for (int i = tid; i < n; i += kLoads * kDistillThreads) {
      uint4 u[kLoads];
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int x = min(i + j * kDistillThreads, n), v = first + x * kN;
        u[j] = x < n && v < live ? ld_stream(row + v) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int x = i + j * kDistillThreads;
        if (x >= n) break;
        const int v = first + x * kN;
        if (v < live) {
          float2 f[kN / 2];
          Vec16<E>::to(u[j], f);
#pragma unroll
          for (int y = 0; y < kN / 2; ++y) {
            f[y].x = v + 2 * y < live ? share(f[y].x) * coef : 0.f;
            f[y].y = v + 2 * y + 1 < live ? share(f[y].y) * coef : 0.f;
          }
          u[j] = Vec16<E>::from(f);
        }
        *reinterpret_cast<uint4 *>(out + v) = u[j];
      }
    }
  } else {
    // (counted from the chunk's start: columns go up to 2^31)
    for (int x = tid; x < e - b; x += kDistillThreads) one(b + x);
  }
  if (!asks) return;
  __syncthreads();
  // The entries' columns.
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int v = in.id[i];
    if (v >= 0) out[v] = Elem<E>::from(g * (mass * share(s[i]) - weight(in.x[i]) * norm));
  }
  const int lane = tid & 31;
  for (int i = tid >> 5; i < sm.n; i += kDistillThreads / 32) {
    const int v = sm.column[i];
    float p = 0.f, count = 0.f;
    for (int y = lane; y < a.k; y += 32) {
      if (a.ids[t * a.ld_ids + y] != v) continue;
      p += weight(teacher_value(a, t * a.ld_teacher + y)) * norm;
      count += 1.f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      p += __shfl_xor_sync(~0u, p, d);
      count += __shfl_xor_sync(~0u, count, d);
    }
    if (lane == 0)
      out[v] = Elem<E>::from(g * (mass * (LISTED ? count : 1.f) * share(sm.score[i]) - p));
  }
}

template <class E, int PER, bool LISTED>
int launch_loss(const DistillArgs &a, cudaStream_t stream) {
  int ctas = 1;
  if (!LISTED) {
    const int64_t wave = resident_ctas(reinterpret_cast<const void *>(distill_loss_kernel<E, PER, LISTED>),
                                       kDistillThreads, 0);
    if (wave == 0) return SATK_ECUDA;
    while (ctas < kMostCluster && a.rows * ctas * 2 <= wave && a.cols / (2 * ctas) >= kLeastChunk)
      ctas *= 2;
  }
  if (a.rows * ctas > INT32_MAX) return SATK_EUNSUPPORTED;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(static_cast<unsigned>(a.rows * ctas));
  config.blockDim = dim3(kDistillThreads);
  config.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  if (cudaLaunchKernelEx(&config, distill_loss_kernel<E, PER, LISTED>, a) != cudaSuccess) {
    cudaGetLastError();
    return SATK_ECUDA;
  }
  return launch_status();
}

template <class E, int PER, bool LISTED>
int launch_grad(DistillArgs a, cudaStream_t stream) {
  // As few chunks as fill the GPU once: each weighs the row's entries for itself.
  const int64_t wave = resident_ctas(reinterpret_cast<const void *>(distill_grad_kernel<E, PER, LISTED>),
                                     kDistillThreads, 0);
  if (wave == 0) return SATK_ECUDA;
  const int64_t least = (a.cols + kChunk - 1) / kChunk, most = (a.cols + kLeastChunk - 1) / kLeastChunk;
  const int64_t chunks = std::max(least, std::min(most, wave / a.rows));
  a.chunk = static_cast<int>(((a.cols + chunks - 1) / chunks + 31) & ~31ll);
  a.chunks = static_cast<int>((a.cols + a.chunk - 1) / a.chunk);
  if (a.rows * a.chunks > INT32_MAX) return SATK_EUNSUPPORTED;
  distill_grad_kernel<E, PER, LISTED>
      <<<static_cast<unsigned>(a.rows * a.chunks), kDistillThreads, 0, stream>>>(a);
  return launch_status();
}

template <class E, int PER>
int launch(const DistillArgs &a, bool grad, bool listed, cudaStream_t stream) {
  if (grad)
    return listed ? launch_grad<E, PER, true>(a, stream) : launch_grad<E, PER, false>(a, stream);
  return listed ? launch_loss<E, PER, true>(a, stream) : launch_loss<E, PER, false>(a, stream);
}

template <class E>
int launch(const DistillArgs &a, bool grad, bool listed, cudaStream_t stream) {
  // Entries of a thread: registers for all of them (four rows of 131071 columns with
  // 2048 entries: gradient 15 us with 8 a thread, 19 with 16).
  if (a.k <= 2 * kDistillThreads) return launch<E, 2>(a, grad, listed, stream);
  if (a.k <= 8 * kDistillThreads) return launch<E, 8>(a, grad, listed, stream);
  return launch<E, SATK_TOPK_MAX_K / kDistillThreads>(a, grad, listed, stream);
}

// The checks and arguments that loss and gradient share.
int checked(DistillArgs &a, const void *logits, int dtype, int64_t rows, int64_t cols,
            int64_t ld_logits, const int32_t *row_ends, const int32_t *ids, int64_t ld_ids,
            int32_t k, const void *teacher, int teacher_dtype, int64_t ld_teacher, int kind,
            int scope, float temperature) {
  const auto known = [](int d) { return d == SATK_F32 || is_16bit(d); };
  if (logits == nullptr || ids == nullptr || teacher == nullptr || !known(dtype) ||
      !known(teacher_dtype) || rows < 0 || rows > INT32_MAX || cols < 0 || cols > INT32_MAX ||
      k < 1 || k > SATK_TOPK_MAX_K || (rows > 1 && (ld_logits < cols || ld_ids < k || ld_teacher < k)) ||
      kind < SATK_TEACHER_LOGITS || kind > SATK_TEACHER_PROBS || scope < SATK_DISTILL_ROW ||
      scope > SATK_DISTILL_LISTED || !std::isfinite(temperature) || !(temperature > 0.f))
    return SATK_EINVAL;
  const float inv_tau = 1.f / temperature;
  if (!std::isfinite(inv_tau * kLog2e) || inv_tau == 0.f) return SATK_EINVAL;
  a = DistillArgs{};
  a.logits = logits;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld_logits;
  a.ends = row_ends;
  a.ids = ids;
  a.ld_ids = ld_ids;
  a.teacher = teacher;
  a.ld_teacher = ld_teacher;
  a.k = k;
  a.teacher_dtype = teacher_dtype;
  a.kind = kind;
  a.inv_tau = inv_tau;
  a.c = inv_tau * kLog2e;
  return SATK_OK;
}

int dispatch(const DistillArgs &a, int dtype, bool grad, int scope, satk_stream_t stream) {
  const bool listed = scope == SATK_DISTILL_LISTED;
  const cudaStream_t s = as_stream(stream);
  if (dtype == SATK_F32) return launch<float>(a, grad, listed, s);
  if (dtype == SATK_BF16) return launch<__nv_bfloat16>(a, grad, listed, s);
  return launch<__half>(a, grad, listed, s);
}

}  // namespace
}  // namespace satk

extern "C" int satk_distill_loss(const void *logits, int dtype, int64_t rows, int64_t cols,
                                 int64_t ld_logits, const int32_t *row_ends, const int32_t *ids,
                                 int64_t ld_ids, int32_t k, const void *teacher, int teacher_dtype,
                                 int64_t ld_teacher, int kind, int scope, float temperature,
                                 float *loss, float *lse, satk_stream_t stream) {
  using namespace satk;
  DistillArgs a;
  const int rc = checked(a, logits, dtype, rows, cols, ld_logits, row_ends, ids, ld_ids, k, teacher,
                         teacher_dtype, ld_teacher, kind, scope, temperature);
  if (rc != SATK_OK) return rc;
  if (loss == nullptr || lse == nullptr) return SATK_EINVAL;
  if (rows == 0) return SATK_OK;
  a.loss = loss;
  a.lse = lse;
  return dispatch(a, dtype, false, scope, stream);
}

extern "C" int satk_distill_grad(const void *logits, int dtype, int64_t rows, int64_t cols,
                                 int64_t ld_logits, const int32_t *row_ends, const int32_t *ids,
                                 int64_t ld_ids, int32_t k, const void *teacher, int teacher_dtype,
                                 int64_t ld_teacher, int kind, int scope, float temperature,
                                 const float *lse, const float *dloss, int32_t dloss_step,
                                 void *grad, int64_t ld_grad, satk_stream_t stream) {
  using namespace satk;
  DistillArgs a;
  const int rc = checked(a, logits, dtype, rows, cols, ld_logits, row_ends, ids, ld_ids, k, teacher,
                         teacher_dtype, ld_teacher, kind, scope, temperature);
  if (rc != SATK_OK) return rc;
  if (lse == nullptr || dloss == nullptr || grad == nullptr || dloss_step < 0 || dloss_step > 1 ||
      (rows > 1 && ld_grad < cols) || (grad == logits && rows > 1 && cols > 0 && ld_grad != ld_logits))
    return SATK_EINVAL;
  if (rows == 0 || cols == 0) return SATK_OK;
  a.lse_in = lse;
  a.dloss = dloss;
  a.dloss_step = dloss_step;
  a.grad = grad;
  a.ld_grad = ld_grad;
  return dispatch(a, dtype, true, scope, stream);
}
