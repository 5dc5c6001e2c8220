// tcgen05.cuh — the fifth-generation tensor-core instructions the prompt
// attention uses: TMEM allocation, matrix descriptors, mma / commit, and TMEM
// loads and stores.
#pragma once

#include "common.cuh"

namespace flint {
namespace tc {

// 512 columns of TMEM (all of an SM's), the address to a shared word; by one warp.
__device__ __forceinline__ void alloc512(uint32_t smem_word) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_word)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc512(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Generic-proxy writes to shared memory -> visible to the tensor core's reads.
__device__ __forceinline__ void fence_smem_to_mma() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulators, A and B both f16 or
// both bf16, M = N = 128, B K-major or MN-major.
constexpr uint32_t inst_desc(bool bf16, bool b_mn_major) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (b_mn_major ? 1u : 0u) << 16 |
         (128u >> 3) << 17 | (128u >> 4) << 24;
}

// Shared-memory matrix descriptor, 128-byte swizzle.  Operands are blocks of
// 64 16-bit elements (128-byte rows, the 16-byte chunk c of row r at c ^ (r % 8)),
// 8 rows a 1024-byte group.  K-major (rows = M or N): `lead` unused.  MN-major
// (rows = K): `lead` is the distance of the next 64 elements of N.
// This is the low word; the high one (group distance, version, swizzle) is the
// same for all.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3fffu) | (lead >> 4) << 16;
}
constexpr uint32_t DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;

// True in one thread of a converged warp.  The products are issued inside
// `if (one_thread())` by a warp whose control flow and operands are uniform:
// they then stay in uniform registers, where the instruction takes them from
// (issued by `if (lane == 0)` with operands of a thread, each mma cost ~200
// cycles of issue, three times its execution).
__device__ __forceinline__ bool one_thread() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

// The same of kind::f8f6f4: A and B E4M3, both K-major.
constexpr uint32_t inst_desc_e4m3() { return 1u << 4 | (128u >> 3) << 17 | (128u >> 4) << 24; }

// D (TMEM) = A B (+ D if add), one step of 32 bytes of K; by one thread.
template <bool E4M3>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t add) {
  if constexpr (E4M3)
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %4, 0;\n"
        "  mov.b64 a, {%1, %5}; mov.b64 b, {%2, %5};\n"
        "  tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p; }" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "r"(DESC_HI)
        : "memory");
  else
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %4, 0;\n"
        "  mov.b64 a, {%1, %5}; mov.b64 b, {%2, %5};\n"
        "  tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p; }" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "r"(DESC_HI)
        : "memory");
}
// A in TMEM (two 16-bit elements a column), kind::f16: one K = 16 step.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t add) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 b; setp.ne.b32 p, %4, 0;\n"
      "  mov.b64 b, {%2, %5};\n"
      "  tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p; }" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(add), "r"(DESC_HI)
      : "memory");
}
// One arrival on `bar` once all of this thread's earlier mma's are complete.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// 32 columns of the warp's 32 TMEM lanes: register i of a lane is column i,
// once wait_ld() has returned.
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
// All of the thread's TMEM loads have arrived.  The registers are not operands
// of the wait: tied to it they were copied, one instruction each, half as many
// as the whole softmax.  Whatever uses them first is volatile itself, which keeps
// it behind this, or goes through arrived().
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void arrived(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace tc
}  // namespace flint
