// satk_tcgen05.cuh -- the fifth-generation tensor core, tensor memory and
// mbarrier operations that the attention kernels use, as inline PTX.
//
// Operands in shared memory are tiles of 128-byte rows in the 128-byte swizzle
// (16-byte chunk c of row r sits at chunk c ^ (r % 8); eight rows form a
// 1024-byte atom, so every tile starts on a 1024-byte boundary):
//   K-major : a row is one M (or N) index, its 128 bytes are 64 consecutive K;
//   MN-major: a row is one K index, its 128 bytes are 64 consecutive M (or N).
// The same tile of keys is read K-major for scores (M = keys, K = columns) and
// MN-major for values (M = columns, K = keys).
//
// Waits are bounded: a wait that has lasted kWaitClocks sets the CTA's `dead`
// word and returns, as every later wait of the CTA then does at once, so all
// roles run through their loops, free what they hold and leave.
#pragma once

#include <cstdint>

#include "satk_device.cuh"

namespace satk {

constexpr long long kWaitClocks = 4000000000ll;  // about two seconds

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// The same without the hardware's suspension: for a thread that polls two.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits until the barrier's phase of this parity has completed.
__device__ __forceinline__ void mbar_wait(uint32_t bar, uint32_t parity, volatile int *dead) {
  if (mbar_test(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_test(bar, parity)) {
    if (*dead != 0) break;
    if (clock64() - t0 > kWaitClocks) *dead = 1;
  }
}

// The same for a role's own copies or MMAs in flight before it leaves: waits
// although the CTA is `dead`, as long as any wait may last.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test(bar, parity) && clock64() - t0 < kWaitClocks) {
  }
}

// Generic-proxy writes to shared memory become visible to the tensor core.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool named_any(int id, int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %3, 0;\n"
      "barrier.cta.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(x ? 1u : 0u)
      : "memory");
  return any != 0;
}

// Register shares of the warpgroups (whole warpgroups, converged).  The shares
// of a CTA add up to at most what it was launched with.
template <int R>
__device__ __forceinline__ void regs_raise() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_lower() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Programmatic dependent launch: a kernel launched with the attribute may start
// before its predecessor in the stream has finished, up to this wait.
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------- async copies --

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// A box of a tensor map (64 columns from `col`, a multiple of 64, of the map's
// rows from `row` on) into consecutive 128-byte rows; rows outside the tensor
// read as zeros.  For a whole converged warp of which the leader issues, as with
// the MMAs below.
__device__ __forceinline__ void tma_box(uint32_t leader, uint32_t dst, const void *map, int col,
                                        int row, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %5, 0;\n"
      "@e cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
      "l"(map), "r"(col), "r"(row), "r"(bar), "r"(leader)
      : "memory");
}

// The 128 bytes around an address into L2 alone.
__device__ __forceinline__ void prefetch_line(const void *src) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(src) : "memory");
}

__device__ __forceinline__ void tma_box3(uint32_t leader, uint32_t dst, const void *map, int col,
                                         int row, int outer, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %6, 0;\n"
      "@e cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
      "l"(map), "r"(col), "r"(row), "r"(outer), "r"(bar), "r"(leader)
      : "memory");
}

// Four rows of a matrix, 64 columns from `col` on (a multiple of 64), into
// consecutive 128-byte rows; the map's box is one row high.  By each thread that
// calls it.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void *map, int col, int4 rows, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(map), "r"(col), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(bar)
      : "memory");
}

// 16 bytes global -> shared; zeros, and no read, when !live.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void cp_async_wait_but_one() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// ------------------------------------------------------------------- tcgen05 --

// Whole warp; the address is written to *slot.
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One lane of a whole converged warp, the same one every time.  MMAs and their
// commits are issued from a branch on it: the compiler knows that such a branch
// has one lane and keeps descriptors in uniform registers, where the instruction
// wants them.  (From a branch on a lane number each MMA costs 20 to 60 cycles
// of moving its operands there.)
__device__ __forceinline__ uint32_t elect_leader() {
  uint32_t leader;
  asm volatile(
      "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n"
      : "=r"(leader));
  return leader;
}

// The barrier's phase gets one arrival when this thread's MMAs so far are done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Instruction descriptor of kind::f16 with fp32 accumulation.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, int M, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor of a 128-byte-swizzled tile: lbo is the distance of
// 64-column blocks along M or N (MN-major only), sbo that of 8-row atoms.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (static_cast<uint64_t>(addr >> 4) & 0x3fff) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
// The same with A in tensor memory: lane = row, a column holds two K values.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(desc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define SATK_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), \
                      "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define SATK_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), \
                      "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])

// 32 lanes x 16 columns: lane l of the warp gets columns [0, 16) of TMEM lane
// (32 (warp % 4) + l).
__device__ __forceinline__ void tmem_ld16(uint32_t (&v)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : SATK_R8(v, 0), SATK_R8(v, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::SATK_I8(v, 0),
      SATK_I8(v, 8), "r"(addr)
      : "memory");
}
// The same for 32 columns, from v[o] on.
template <int LEN>
__device__ __forceinline__ void tmem_ld32(uint32_t (&v)[LEN], const int o, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : SATK_R8(v, o), SATK_R8(v, o + 8), SATK_R8(v, o + 16), SATK_R8(v, o + 24)
      : "r"(addr)
      : "memory");
}
template <int LEN>
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[LEN], const int o) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::SATK_I8(v, o),
      SATK_I8(v, o + 8), SATK_I8(v, o + 16), SATK_I8(v, o + 24), "r"(addr)
      : "memory");
}
// 16 lanes x 2 C columns: lanes 0-15 of the warp get columns [0, C) of their
// TMEM lane, lanes 16-31 columns [C, 2 C) of TMEM lanes 0-15 of the quarter (an
// M = 64 accumulator keeps its rows 16 w .. 16 w + 15 there).
template <int C>
__device__ __forceinline__ void tmem_ld_half(uint32_t (&v)[C], uint32_t addr) {
  static_assert(C == 8 || C == 16 || C == 32, "columns per half");
  if constexpr (C == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
        : SATK_R8(v, 0)
        : "r"(addr)
        : "memory");
  } else if constexpr (C == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16], 16;"
        : SATK_R8(v, 0), SATK_R8(v, 8)
        : "r"(addr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;"
        : SATK_R8(v, 0), SATK_R8(v, 8), SATK_R8(v, 16), SATK_R8(v, 24)
        : "r"(addr)
        : "memory");
  }
}

// 32 lanes x 8 columns of tensor memory.
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::SATK_I8(v, 0),
               "r"(addr)
               : "memory");
}

// 32 columns of 16 lanes, eight columns a step: a thread gets columns 2 (l % 4) and
// the next one of lanes l / 4 and l / 4 + 8, for its lane l of the warp.
__device__ __forceinline__ void tmem_ld_pairs(uint32_t (&v)[32], const int o, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : SATK_R8(v, o), SATK_R8(v, o + 8)
      : "r"(addr)
      : "memory");
}
// The same of 16 columns.
__device__ __forceinline__ void tmem_ld_pairs_half(uint32_t (&v)[32], const int o, uint32_t addr) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : SATK_R8(v, o)
               : "r"(addr)
               : "memory");
}
// The same places of 16 columns that hold two 16-bit values each.
__device__ __forceinline__ void tmem_st_packed(uint32_t addr, const uint32_t (&v)[16], const int o) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::SATK_I8(v, o),
               "r"(addr)
               : "memory");
}

// MMAs with descriptors whose upper words are all the same (atoms of eight rows are
// 1024 bytes apart): the lower words are what changes, a constant away from one
// uniform register.  What the one issuing thread does between MMAs counts: 64-bit
// sums cost 50 cycles an MMA, a branch 40 to 60, a satisfied barrier wait 90, a
// commit or a fence nothing, while an MMA of 64 columns runs for 32 to 50.  So the
// issuing loops are straight lines: panel counts are constants, what not every
// shape has is predicated, rings wrap by selects.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3fff) | (lbo >> 4) << 16;
}
__device__ __forceinline__ void mma_ss_low(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool more) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "setp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(more ? 1u : 0u), "r"(kDescHigh)
      : "memory");
}
// The same only where `on`: a predicate, not a branch.
__device__ __forceinline__ void mma_ss_low_if(bool on, uint32_t d, uint32_t a, uint32_t b, uint32_t desc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 x, y;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "setp.ne.u32 e, %4, 0;\nsetp.eq.u32 p, 0, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(on ? 1u : 0u), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts_low_if(bool on, uint32_t d, uint32_t a, uint32_t b, uint32_t desc) {
  asm volatile(
      "{\n.reg .pred p, e;\n.reg .b64 y;\nmov.b64 y, {%2, %5};\n"
      "setp.ne.u32 e, %4, 0;\nsetp.eq.u32 p, 0, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(on ? 1u : 0u), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void tc_commit_if(bool on, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(on ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts_low(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool more) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 y;\nmov.b64 y, {%2, %5};\n"
      "setp.ne.u32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"(more ? 1u : 0u), "r"(kDescHigh)
      : "memory");
}

}  // namespace satk
