// Fifth-generation tensor core instructions (tcgen05) as inline PTX: tensor
// memory, matrix products with fp32 sums, and their completion on mbarriers.
#pragma once

#include <stdint.h>

#include "tma.cuh"

namespace fp8q {

__device__ __forceinline__ void tmem_alloc(uint32_t* smem_result, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_result)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive columns of this warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// Wait for this warp's loads; r (of the last one) is only then defined.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle, in two halves: the start
// address and leading byte offset (multiples of 16) make the low one, the
// stride byte offset the high one.  An operand further on has a low half
// larger by bytes / 16, so that the products of a loop share one base.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | ((lead >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride) { return (stride >> 4) | (1u << 14) | (2u << 29); }
// Instruction descriptor of kind::f16 with f16 operands and fp32 sums;
// b_mn: B is stored with its N dimension consecutive.
__host__ __device__ constexpr uint32_t f16_idesc(int m, int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// d (tensor memory) = a * b, or += where accumulate; issued by one thread.
// A and B by the low halves of their descriptors, which share the high half.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc),
      "r"((uint32_t)accumulate)
      : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc),
      "r"((uint32_t)accumulate)
      : "memory");
}
// Block-scaled products: each 32 elements along K of a row of A and B are
// scaled by an E8M0 byte in tensor memory.  Scales of 128 rows x 128 elements
// are four columns of words, word j of lane i (of each 32) being row 32 j + i's
// four bytes; sf_copy brings them there from 512 bytes of shared memory, row
// 32 j + i at byte 16 i + 4 j.  A product takes 64 elements of 4 bits (bytes
// 2 s and 2 s + 1 of the words, s = 0 or 1) or 32 of 8 bits (byte s).
__host__ __device__ constexpr uint32_t mx_idesc(bool four, int a_format, int b_format, int m, int n) {
  // the E8M0 scales' bit, M and N; operand formats: E2M1 is 1 in the 4-bit kind, E4M3 0 and E5M2 1 in the 8-bit one
  return (1u << 23) | ((uint32_t)(four ? 1 : a_format) << 7) | ((uint32_t)(four ? 1 : b_format) << 10) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// The same with step s of a word's bytes chosen for both operands.
template <bool F4>
__host__ __device__ constexpr uint32_t mx_idesc_step(uint32_t idesc, int s) {
  return idesc | ((uint32_t)(F4 ? 2 * s : s) << 4) | ((uint32_t)(F4 ? 2 * s : s) << 29);
}
// Shared-memory descriptor of sf_copy's 32 rows of 16 bytes (no swizzle, eight
// rows every 128 bytes).
__device__ __forceinline__ uint64_t sf_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((128u >> 4) | (1u << 14)) << 32);
}
template <int CTAS>
__device__ __forceinline__ void sf_copy(uint32_t tmem, uint64_t desc) {
  if (CTAS == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
#define FP8Q_MX_MMA(group, kind)                                                                               \
  asm volatile(                                                                                                \
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %7, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n" \
      " tcgen05.mma.cta_group::" group ".kind::" kind " [%0], a, b, %4, [%5], [%6], p;\n}" ::"r"(d),           \
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sf_a), "r"(sf_b), "r"((uint32_t)accumulate)               \
      : "memory")
template <bool F4, int CTAS>
__device__ __forceinline__ void mma_mx(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                       uint32_t sf_a, uint32_t sf_b, bool accumulate) {
  if (F4 && CTAS == 1) FP8Q_MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
  if (F4 && CTAS == 2) FP8Q_MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
  if (!F4 && CTAS == 1) FP8Q_MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
  if (!F4 && CTAS == 2) FP8Q_MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
}
#undef FP8Q_MX_MMA
// One arrival on bar once every product issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ---- pairs of CTAs (cta_group::2): a product of 256 rows, 128 in each CTA's
// tensor memory, with each CTA's shared memory holding its rows of A and half
// the rows of B.  The even CTA of the pair issues copies and products.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_result, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(smem_result)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
// One arrival on each CTA's barrier at bar's place.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The even CTA's barrier at bar's place, as an address of the cluster.
__device__ __forceinline__ uint32_t lead_bar(const uint64_t* bar) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(bar)));
  return a;
}
// One arrival on a barrier of the pair for shared memory that the arriving warp
// wrote for the pair's products, after a proxy fence of each lane.  The arrival
// releases at CTA scope, the default.  From the odd CTA to the even one, whose
// thread issues the products, PTX's memory model promises the order of writes only
// for a release (and an acquire) of cluster scope: that the products see the odd
// CTA's scales is what the hardware does, whose proxy fence is over when the
// writes are in shared memory, and not what the model says.  The acquire would
// cost nothing, but a release of cluster scope waits for a round trip to L2 and for
// the thread's loads in flight.  8192 x 8192 x 8192 in 4 bits 157 us (8 bits 325);
// with such a release by the warps that bring scales 1.7 times as long as without,
// by one warp that they tell 342 (880), by four in turn 181 (368), by three in turn
// for two blocks at a time, scales' stages free again once they are copied, 168 (332).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same where all that has to come before are tensor-memory loads, which the
// thread has waited for: without a release, which would wait for its stores to
// global memory as well.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Tile into this CTA's shared memory, its bytes counted on a barrier of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// One lane of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// mbar_wait for warps that share the SM's issue slots with busy ones: the
// clock is read only every 64th try (each try suspends the warp for a while
// by itself; one with a time hint becomes a loop of sleeps, which wakes late).
__device__ __forceinline__ bool mbar_wait_lean(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long deadline = clock64() + kWaitCycles;
  do {
#pragma unroll 1
    for (int n = 0; n < 64; ++n)
      if (mbar_try_wait(bar, parity)) return true;
  } while (clock64() < deadline);
  return false;
}

template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace fp8q
