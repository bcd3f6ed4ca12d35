// Fifth-generation tensor cores: the PTX that the prompt attention kernel
// uses (tcgen05.mma with its accumulators, and the softmax weights as A
// operand, in tensor memory).
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace tc {

// One thread of the warp, which the compiler knows to be alone in the branch:
// operands of tensor and copy instructions then go to uniform registers once,
// not in a loop over the lanes.  All lanes call together.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Takes over a CTA of this grid that has not started yet (whose blockIdx.x the
// 16 bytes at `at` then hold), or learns that there is none; completes on `bar`.
// Not called again once there is none.
__device__ __forceinline__ void steal_cta(uint32_t at, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(at),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ int stolen_cta(uint32_t at) {  // -1: none
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(at)
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// Tensor memory: 128 lanes of 512 32-bit columns a SM; an address is (lane
// << 16) | column, and a warp reaches the 32 lanes of its rank modulo 4.
__device__ __forceinline__ void alloc(uint32_t result, uint32_t columns) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void dealloc(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrives on `bar` when every MMA issued so far by this thread has completed.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Descriptor of a 16-bit operand in shared memory in the 128-byte swizzle
// (8 rows of 128 bytes an atom).  K-major (rows of K): atoms `sbo` bytes
// apart along the rows.  MN-major (rows of the other dimension, 64 of it a
// row): `sbo` between atoms along K, `lbo` between groups of 64.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, 128 x N tiles with f32 accumulators.
constexpr uint32_t instr_desc(bool bf16, int n, bool b_mn_major, bool negate_a) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (negate_a ? 1u << 13 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}

#define PKV_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
                     "=r"(r[i + 6]), "=r"(r[i + 7])
#define PKV_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
                     "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this thread's lane (thread i of the warp: lane 32 (warp % 4) + i).
__device__ __forceinline__ void ld32(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : PKV_R8(r, 0), PKV_R8(r, 8), PKV_R8(r, 16), PKV_R8(r, 24)
      : "r"(at));
}
__device__ __forceinline__ void ld8(uint32_t* r, uint32_t at) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];" : PKV_R8(r, 0) : "r"(at));
}
// 64 columns of 16 lanes (those from the address'): thread i has columns 8k + 2
// (i % 4), + 1 of lanes i / 4 (r[4k], r[4k + 1]) and i / 4 + 8 (r[4k + 2], r[4k + 3]).
__device__ __forceinline__ void ld16x64(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : PKV_R8(r, 0), PKV_R8(r, 8), PKV_R8(r, 16), PKV_R8(r, 24)
      : "r"(at));
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::PKV_I8(r, 0),
      PKV_I8(r, 8), PKV_I8(r, 16), PKV_I8(r, 24), "r"(at)
      : "memory");
}

__device__ __forceinline__ void st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::PKV_I8(r, 0),
      PKV_I8(r, 8), "r"(at)
      : "memory");
}

__device__ __forceinline__ void st8(uint32_t at, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::PKV_I8(r, 0), "r"(at)
               : "memory");
}

#undef PKV_R8
#undef PKV_I8

}  // namespace tc
}  // namespace pkv
