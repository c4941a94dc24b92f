// PTX of the tcgen05 kernels (gemm_tc.cu, attn.cu, linear8_tc.cu): mbarriers with bounded waits, TMA copies, tensor
// memory loads and stores, matrix descriptors.
#pragma once

#include "moe_internal.cuh"
#include "tensor_map.cuh"

namespace moe {

constexpr long long kTimeoutCycles = 4000000000LL;  // ~2 s at 2 GHz

__device__ __forceinline__ uint32_t su32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(su32(b)), "r"(count));
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(su32(b)), "r"(bytes) : "memory");
}
// A waiting thread is suspended in hardware until the phase completes (or the hint, 1 ms, runs
// out) instead of re-issuing the test: the compute warps waiting on their stages would otherwise
// take issue slots from the single-thread MMA and copy loops on their SM sub-partitions.
template <bool CL = false>
__device__ __forceinline__ bool mbar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  if constexpr (CL)   // barriers the other CTA of a pair arrives on (remote arrivals, multicast commits)
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000000;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000000;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
  return ok != 0;
}
// Bounded wait: false if the CTA aborted or this wait expired (then the abort flag is set and the
// code goes to the translation unit's device error word).
template <bool CL = false>
__device__ __forceinline__ bool mbar_wait(uint64_t *b, uint32_t parity, volatile int *abort_flag, int code, int *error) {
  if (mbar_try<CL>(b, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try<CL>(b, parity)) return true;
    if ((it & 7) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kTimeoutCycles) {
        *abort_flag = 1;
        atomicExch(error, code);
        return false;
      }
    }
  }
}

// The same on a shared-memory address (no generic address arithmetic on a single thread's critical path).
__device__ __forceinline__ bool mbar_try_at(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(addr), "r"(parity)
               : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_at(uint32_t addr, uint32_t parity, volatile int *abort_flag, int code, int *error) {
  if (mbar_try_at(addr, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_at(addr, parity)) return true;
    if ((it & 7) == 0) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kTimeoutCycles) {
        *abort_flag = 1;
        atomicExch(error, code);
        return false;
      }
    }
  }
}

// ---- CTA pairs (clusters of two): addresses in the peer CTA, remote arrivals, cluster barrier
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// shared::cluster address of the same shared-memory location in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t map_to_rank(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(su32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
          su32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(su32(bar))
      : "memory");
}

// Bring a weight box into L2 ahead of its shared-memory copy (no barrier, no shared memory).
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(su32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_commit_at(uint32_t addr) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(addr) : "memory");
}
// pairs: completion of the pair's MMAs issued so far, signalled on `bar` in both CTAs / in this one
__device__ __forceinline__ void tc_commit_pair(uint64_t *bar) {
  const uint16_t both = 3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
          su32(bar)),
      "h"(both)
      : "memory");
}
__device__ __forceinline__ void tc_commit_pair_local(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(su32(bar))
               : "memory");
}

// A from shared memory (16-bit weights)
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The eight MMAs of one 128-wide K block (A from tensor memory), in one statement: the first
// accumulates only when `acc` is set, the others always; MMA j reads A columns a + 8j and the
// B descriptor advanced by j's start offset (16-byte units: 2 per 16-wide step inside a 64-wide
// swizzle atom column, half16 to the next column block).  The offsets are added to the low word
// only: the start-address field cannot carry (shared addresses stay below 256 KB).
#define MOE_TC_MMA_KBLOCK(GROUP)                                                                                  \
  asm volatile(                                                                                                   \
      "{\n .reg .pred p, t;\n .reg .b32 a1, bl1;\n .reg .b64 bd;\n"                                            \
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, %5, %5;\n"                                                       \
      " mov.b64 bd, {%2, %3};\n tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [%1], bd, %4, p;\n"             \
      " add.u32 a1, %1, 8;\n add.u32 bl1, %2, 2;\n mov.b64 bd, {bl1, %3};\n"                                  \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 16;\n add.u32 bl1, %2, 4;\n mov.b64 bd, {bl1, %3};\n"                                 \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 24;\n add.u32 bl1, %2, 6;\n mov.b64 bd, {bl1, %3};\n"                                 \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 32;\n add.u32 bl1, %2, %6;\n mov.b64 bd, {bl1, %3};\n"                                \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 40;\n add.u32 bl1, %2, %7;\n mov.b64 bd, {bl1, %3};\n"                                \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 48;\n add.u32 bl1, %2, %8;\n mov.b64 bd, {bl1, %3};\n"                                \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      " add.u32 a1, %1, 56;\n add.u32 bl1, %2, %9;\n mov.b64 bd, {bl1, %3};\n"                                \
      " tcgen05.mma.cta_group::" GROUP ".kind::f16 [%0], [a1], bd, %4, t;\n"                                     \
      "}\n" ::"r"(d), "r"(a), "r"(bl), "r"(bh), "r"(idesc), "r"(acc), "n"(HALF16), "n"(HALF16 + 2), "n"(HALF16 + 4), \
      "n"(HALF16 + 6)                                                                                             \
      : "memory")
template <int HALF16, bool PAIR>
__device__ __forceinline__ void tc_mma_kblock_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  const uint32_t bl = uint32_t(b), bh = uint32_t(b >> 32);
  if constexpr (PAIR) MOE_TC_MMA_KBLOCK("2");   // M = 256: A rows and B columns from both CTAs of the pair
  else MOE_TC_MMA_KBLOCK("1");
}
#undef MOE_TC_MMA_KBLOCK

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFFu);          // start address
  d |= uint64_t(1) << 16;                          // leading byte offset (unused with swizzle)
  d |= uint64_t(1024 >> 4) << 32;                  // stride byte offset
  d |= uint64_t(1) << 46;                          // descriptor version
  d |= uint64_t(2) << 61;                          // SWIZZLE_128B
  return d;
}

// Instruction descriptor, kind::f16: fp32 D, A/B f16 (0) or bf16 (1), both K-major.
__host__ __device__ constexpr uint32_t idesc_f16(int is_bf16, int M, int N) {
  return (1u << 4) | (uint32_t(is_bf16) << 7) | (uint32_t(is_bf16) << 10) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

}  // namespace moe
