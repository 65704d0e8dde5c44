// ptx.cuh -- thin inline-PTX wrappers for sm_103a: mbarrier, TMA (cp.async.bulk.tensor),
// tcgen05 (TMEM alloc / MMA / commit / ld / st), cluster barriers, and bounded waits.
//
// Every wait in this library is bounded: it gives up after kWaitLimitNs of %globaltimer time,
// raises the CTA's abort flag and reports DSA_ERR_TIMEOUT through the caller's status word, so a
// logic error can never hang the GPU.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#define DSA_DEV __device__ __forceinline__

namespace dsa {

#ifdef DSA_TEST_HOOKS
// Test build (libdsa_testhooks.so): a short limit, so that a test can make a wait run out
// quickly and check that the kernel reports it and frees what it holds.
constexpr uint64_t kWaitLimitNs = 20ull * 1000ull * 1000ull;    // 20 ms per wait
#else
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;  // 1 s per wait
#endif
constexpr uint32_t kSuspendHintNs = 20000u;                       // sleep per try_wait

enum : int { kStatusOk = 0, kStatusDeviceCheck = 4, kStatusTimeout = 5 };

DSA_DEV void report(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

DSA_DEV uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

DSA_DEV uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

DSA_DEV uint32_t elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(pred));
  return pred;
}

// ---------------------------------------------------------------- programmatic dependent launch

// Wait until the preceding kernel in the stream has completed and its memory is visible (a no-op
// when the kernel was launched without programmatic stream serialisation).
DSA_DEV void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Allow the kernel launched after this one with programmatic stream serialisation to begin
// scheduling its CTAs once every CTA of this grid has passed here (or exited).
DSA_DEV void griddep_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- mbarrier

DSA_DEV void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

DSA_DEV void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

DSA_DEV void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

DSA_DEV void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// One potentially-blocking test of phase `parity`: the thread is suspended (issuing nothing)
// until the phase completes or the hinted time (ns) passes.
DSA_DEV bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
      : "memory");
  return ok != 0;
}

// Non-blocking test of phase `parity`.
DSA_DEV bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Non-blocking test of phase `parity` with acquire semantics at cluster scope (for phases completed
// by another CTA's asynchronous stores).
DSA_DEV bool mbar_test_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// As mbar_try_wait, with acquire semantics at cluster scope: for phases completed by arrivals
// of another CTA of the cluster that released its own shared::cluster stores.
DSA_DEV bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
      : "memory");
  return ok != 0;
}

// Arrive on an mbarrier of another CTA of the cluster (shared::cluster address) without ordering
// this thread's earlier memory operations: for signals whose only precondition is that values
// this thread loaded have been consumed (an in-order thread issues the arrive after them).
DSA_DEV void mbar_arrive_remote_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Asynchronous 16-byte store into the shared memory of a CTA of the cluster; its completion is
// counted (16 bytes) on that CTA's mbarrier `remote_bar` (both shared::cluster addresses).
DSA_DEV void st_async_v4(uint32_t cluster_addr, uint4 v, uint32_t remote_bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(
          cluster_addr),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(remote_bar)
      : "memory");
}

// Asynchronous 4-byte store into the shared memory of a CTA of the cluster, counted (4 bytes) on
// that CTA's mbarrier `remote_bar`.
DSA_DEV void st_async_b32(uint32_t cluster_addr, uint32_t v, uint32_t remote_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                   cluster_addr),
               "r"(v), "r"(remote_bar)
               : "memory");
}

// Bounded wait for phase `parity` of `bar`.  Returns false (and raises *abort) when the limit
// runs out or another thread of the CTA already aborted.
template <bool kCluster = false>
DSA_DEV bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  auto try_once = [&]() {
    return kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  };
  if (try_once()) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
      if (try_once()) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > kWaitLimitNs) {
      *abort = 1;
      report(status, kStatusTimeout);
      return false;
    }
  }
}

// As mbar_wait, kept out of line, for waits whose phase has usually completed: a test (17 cycles
// against 51 of a try_wait) stands before the call.
static __device__ __noinline__ bool mbar_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                   int* status) {
  if (*abort) return false;
  return mbar_wait(bar, parity, abort, status);
}
DSA_DEV bool mbar_wait_fast(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_test(bar, parity) || mbar_wait_slow(bar, parity, abort, status);
}

// Bounded wait of a whole warp, which is converged again after it.
DSA_DEV void warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  mbar_wait_fast(bar, parity, abort, status);
  __syncwarp();
}

// mbar_wait_fast for the warp that issues a CTA's (or a CTA pair's, kPair) MMAs.  After a wait that gave up it goes on
// through its program, and commits on the release of parts that never came; a loader that took such a release
// would arm a barrier whose bytes are outstanding, one arrival too many.  So it tells the pair's other CTA
// (rank 1) too and stays here until every loader has noticed (a waiting thread looks at the abort flag every
// four suspensions, 80 us) and left.  (An issue that can be called off instead, by a predicate that changes, took
// a third longer for a whole call.)
template <bool kPair>
static __device__ __noinline__ bool mbar_wait_issue_slow(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                         int* status) {
  if (!*abort && mbar_wait(bar, parity, abort, status)) return true;
  if (kPair)
    asm volatile(
        "{\n .reg .u32 a;\n mapa.shared::cluster.u32 a, %0, 1;\n st.volatile.shared::cluster.u32 [a], 1;\n}\n" ::"r"(
            smem_u32(const_cast<const int*>(abort)))
        : "memory");
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000u) {
  }
  return false;
}
template <bool kPair>
DSA_DEV bool mbar_wait_issue(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_test(bar, parity) || mbar_wait_issue_slow<kPair>(bar, parity, abort, status);
}

// Bounded wait that does not give up when the CTA has aborted: for draining asynchronous copies
// that were issued and will complete (their bytes exist) before their destination is reused or
// the CTA exits.
DSA_DEV bool mbar_wait_drain(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      report(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------- TMA

DSA_DEV void prefetch_tmap(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// 2-D tiled load of one box into shared memory, completing bytes on `bar`.
// L2 policy for data that is read once: its lines are the first to be replaced, so a stream
// larger than L2 does not push out code and the small tensors other CTAs still need.
DSA_DEV uint64_t l2_policy_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
DSA_DEV void tma_load_2d_hint(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y,
                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
DSA_DEV void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

DSA_DEV void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Bulk prefetch of `bytes` (a multiple of 16, 16-byte aligned) of global memory into L2.
DSA_DEV void prefetch_l2_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(p)),
               "r"(bytes)
               : "memory");
}

// Four rows (y0..y3) of one column box (x) of a 2-D map whose box is one row high.
DSA_DEV void tma_gather4(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y0, int y1,
                         int y2, int y3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y0), "r"(y1), "r"(y2),
      "r"(y3)
      : "memory");
}

// Named barrier over `nthreads` threads (a multiple of 32); blocks in hardware.
DSA_DEV void named_barrier(uint32_t id, uint32_t nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// Named barrier that also reduces a predicate: every participating thread gets the AND of `v`
// over all of them, so a group can decide together (e.g. to leave a loop) and never strand a
// member at a later barrier.
DSA_DEV bool named_barrier_and(uint32_t id, uint32_t nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(nthreads)
      : "memory");
  return r != 0;
}

DSA_DEV void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------- tcgen05

DSA_DEV void tmem_alloc(uint32_t* result_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(result_smem)),
               "r"(ncols)
               : "memory");
}
DSA_DEV void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
DSA_DEV void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
DSA_DEV void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
DSA_DEV void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit inputs (kind::f16), fp32 accumulate.
DSA_DEV void mma_f16_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Same with A read from tensor memory.
DSA_DEV void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 8-bit float inputs (kind::f8f6f4), fp32 accumulate.
DSA_DEV void mma_f8_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MXFP8 (kind::mxf8f6f4, e4m3 A/B, E8M0 scale per 32 K elements), fp32 accumulate.  One MMA
// covers K = 32, i.e. one scale per row of A and per column of B, read from tensor memory:
// sfa holds A's scales (row r at lane r, column sfa + r/32), sfb B's (column n at lane
// 32*q + n%32 of every lane quadrant q, column sfb + n/32); the instruction descriptor picks
// the byte of each 32-bit cell.
DSA_DEV void mma_mx_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                       uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Arrive once on `bar` when every MMA issued so far by this thread has completed.
DSA_DEV void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Instruction descriptor, kind::f16 with bf16 A/B and fp32 D.  b_mn_major selects an MN-major
// (N-contiguous) B operand.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool b_mn_major = false) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// kind::f8f6f4 with e4m3 A/B and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | (0u << 7) | (0u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// kind::mxf8f6f4 with e4m3 A/B, E8M0 scales (bit 23), fp32 D; sf_a / sf_b select the byte of
// the 32-bit scale cell used for A and for B.
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int M, int N, int sf_a, int sf_b) {
  return ((uint32_t)sf_b << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24) | ((uint32_t)sf_a << 29);
}

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major operands: rows of 128 B, 8-row
// groups 1024 B apart (sbo = 1024).  MN-major operands: lbo = distance between 64-element column
// blocks, sbo = distance between 8-row groups along K.
// K-major operand with 64-byte rows, 64-byte swizzle (16-byte chunk c of row r stored at chunk
// c ^ ((r >> 1) & 3)); 8-row groups are sbo (512) bytes apart.
DSA_DEV uint64_t sdesc_sw64(uint32_t saddr, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;  // leading byte offset: unused for swizzled K-major
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  d |= (uint64_t)4 << 61;  // 64-byte swizzle
  return d;
}
DSA_DEV uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// tcgen05.ld, 32 lanes x 32 bit, N consecutive columns per thread.
DSA_DEV void tmem_ld_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}

DSA_DEV void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

DSA_DEV void tmem_ld_x32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

DSA_DEV void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

DSA_DEV void tmem_st_x1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}

DSA_DEV void tmem_st_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

DSA_DEV void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

DSA_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The one-CTA forms for a whole converged warp: they act in the lane whose `issuer` is not 0 (one,
// always the same), so that their operands stay in uniform registers (see the two-CTA forms).
DSA_DEV void mma_f16_ss_by(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                           uint32_t accumulate, uint32_t issuer) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issuer)
      : "memory");
}
DSA_DEV void mma_f16_ts_by(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                           uint32_t accumulate, uint32_t issuer) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issuer)
      : "memory");
}
DSA_DEV void mma_commit_by(uint64_t* bar, uint32_t issuer) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar)),
      "r"(issuer)
      : "memory");
}

// ---------------------------------------------------------------- two-CTA tcgen05 (cta_group::2)
//
// The CTA pair of a cluster (ranks 2i, 2i + 1) as one MMA unit: the even CTA issues, each CTA
// holds its half of A's rows and of B's rows (columns of D) at the same shared-memory offset, and
// its half of D's rows in its own tensor memory.  With M = 128 a CTA has 64 rows of D: lane l < 64
// holds columns 0 .. N/2 - 1 of row l, lane 64 + l columns N/2 .. N - 1 of the same row (checked
// with integer operands for N = 32 .. 256, K-major and MN-major B).  Measured, issued back to back:
// 49 cycles an instruction for N <= 128, 64 for N = 256.

DSA_DEV void tmem_alloc2(uint32_t* result_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(result_smem)),
               "r"(ncols)
               : "memory");
}
DSA_DEV void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
DSA_DEV void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
// These two are executed by a whole converged warp and act in the lane whose `issuer` is not 0 (one,
// always the same): with no divergent branch around them their operands stay in uniform registers,
// which the instruction reads (behind an `if (lane == 0)` each MMA took about 90 cycles to issue).
DSA_DEV void mma2_f16_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                         uint32_t accumulate, uint32_t issuer) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(issuer)
      : "memory");
}
// Arrive once on `bar` of both CTAs of the pair (same offset) when every MMA issued so far by this
// thread has completed.
DSA_DEV void mma2_commit_both(uint64_t* bar, uint32_t issuer) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3), "r"(issuer)
      : "memory");
}
// 2-D tiled load into this CTA's shared memory that completes bytes on an mbarrier of either CTA of
// the pair (shared::cluster address).
DSA_DEV void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(x), "r"(y)
      : "memory");
}
// Arrive on an mbarrier of either CTA of the pair for data that the tensor cores read from this
// CTA's own shared memory (or tensor memory): this thread's fences toward the async proxy have
// ordered it already, so the arrival releases at CTA scope only.  A release at cluster scope waits
// for every earlier access of the thread to be performed cluster-wide (measured: 2,000 cycles).
DSA_DEV void mbar_arrive_pair(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster)
               : "memory");
}

// ---------------------------------------------------------------- cluster

DSA_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
DSA_DEV uint32_t cluster_nrank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
DSA_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Split cluster barrier: arrive (release) now, wait (acquire) later.
DSA_DEV void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
DSA_DEV void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in CTA `rank` of the cluster (shared::cluster window).
DSA_DEV uint32_t map_cluster(const void* local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  return r;
}
DSA_DEV uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
DSA_DEV uint2 ld_cluster_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
DSA_DEV void st_cluster_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
// Bulk copy of `bytes` (multiple of 16) from this CTA's shared memory to the shared memory of a
// CTA of the cluster (shared::cluster address), counted on that CTA's mbarrier `remote_bar`.
// The source must have been made visible to the async proxy (fence_proxy_async_smem).
DSA_DEV void bulk_copy_to_cluster(uint32_t dst_cluster, const void* src, uint32_t bytes,
                                  uint32_t remote_bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst_cluster), "r"(smem_u32(src)), "r"(bytes), "r"(remote_bar)
      : "memory");
}
DSA_DEV void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until every committed bulk copy of this thread has finished reading its source.
DSA_DEV void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
DSA_DEV uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ---------------------------------------------------------------- cluster launch control

// Ask for a block of this grid that has not started: its index, or that there is none, arrives as 16
// bytes in shared memory, counted on `bar`.  The grid's remaining blocks go to whoever asks first.  Not
// to be asked again after the answer that there is none.
DSA_DEV void clc_try_cancel(void* response, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(response)),
      "r"(smem_u32(bar))
      : "memory");
}
// The x index of the block in an answer, or -1: none.
DSA_DEV int clc_block(const void* response) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n ld.shared.b128 r, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(response))
      : "memory");
  return ok ? (int)x : -1;
}

// ---------------------------------------------------------------- misc

// A shared-memory matrix descriptor moved by a constant (the address field cannot carry: every operand
// lies below 256 KiB).
DSA_DEV uint64_t desc_at(uint64_t d, int bytes) {
  uint32_t lo = (uint32_t)d, hi = (uint32_t)(d >> 32);
  lo += (uint32_t)(bytes >> 4);
  return ((uint64_t)hi << 32) | lo;
}

// 32 bytes to global memory, a full sector (32-byte aligned).
DSA_DEV void st_global_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Largest, and smallest, of three (a NaN loses), one instruction.
DSA_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
DSA_DEV float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^x with the hardware approximation (flush-to-zero; 2^-inf = 0).  The weights are rounded to
// bf16 right after, so its ~2-ulp fp32 error is far below what the output keeps.
DSA_DEV float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
DSA_DEV uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Two bf16 with what is not finite set to zero.
DSA_DEV uint32_t finite_bf16x2(uint32_t e) {
  if ((e & 0x7f80u) == 0x7f80u) e &= 0xffff0000u;
  if ((e & 0x7f800000u) == 0x7f800000u) e &= 0xffffu;
  return e;
}
// Two fp32 products with one factor (a packed multiplication: one instruction for both).
DSA_DEV float2 mul2(float2 a, float s) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mul.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(s));
  return d;
}
// a * s + t on two values, and the sum of two pairs: one packed instruction each.
DSA_DEV float2 fma2(float2 a, float s, float t) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(s), "f"(t));
  return d;
}
DSA_DEV float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Order-preserving map of an fp32 score to uint32 (larger score -> larger key); -0.0 and +0.0
// map to the same key.  Key 0 is reserved for "not a candidate" (no finite score maps there).
DSA_DEV uint32_t score_key(float s) {
  uint32_t b = __float_as_uint(s);
  if ((b << 1) == 0) b = 0;  // fold -0.0 onto +0.0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// Inverse of score_key (for keys of finite scores).
DSA_DEV float key_score(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

}  // namespace dsa
