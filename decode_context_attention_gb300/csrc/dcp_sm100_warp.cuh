// dcp_sm100_warp.cuh -- wrappers over the sm_100-family PTX that the chunk kernels
// (dcp_chunk_attention_tc.cu, dcp_chunk_weights_tc.cu) add to dcp_sm100.cuh:
// products issued by a converged warp, wide tensor-memory loads, register splits.
#pragma once

#include "dcp_sm100.cuh"

namespace dcp {
namespace sm100 {

// Products and commits, called by a whole converged warp whose leader (elect.sync,
// the same thread every time) issues: operands that are uniform over the warp then
// stay in uniform registers, which the instructions take, where a single
// thread's registers have to be moved there one by one.
__device__ __forceinline__ void mma_commit_warp(uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
        : "memory");
}

// Four products in a row, their operands A_STEP and B_STEP apart (in the descriptors'
// 16-byte units, or TMEM columns).  The descriptors are put together here, from
// their low words: held across a loop, the 64-bit descriptors of every step took
// more registers than the issuing warp has.
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void mma_ss4_warp(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                             uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 x, y;\n .reg .b64 a, b;\n"
        " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %6, 0;\n setp.eq.b32 t, 0, 0;\n"
        " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n"
        " add.u32 x, %1, %7;\n add.u32 y, %3, %8;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n"
        " add.u32 x, x, %7;\n add.u32 y, y, %8;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n"
        " add.u32 x, x, %7;\n add.u32 y, y, %8;\n mov.b64 a, {x, %2};\n mov.b64 b, {y, %4};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accum), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void mma_ts4_warp(uint32_t d, uint32_t a_tmem, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                             uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p, t, e;\n .reg .b32 x, y;\n .reg .b64 b;\n"
        " elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"
        " mov.b64 b, {%2, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n"
        " add.u32 x, %1, %6;\n add.u32 y, %2, %7;\n mov.b64 b, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
        " add.u32 x, x, %6;\n add.u32 y, y, %7;\n mov.b64 b, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
        " add.u32 x, x, %6;\n add.u32 y, y, %7;\n mov.b64 b, {y, %3};\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n}" ::"r"(d),
        "r"(a_tmem), "r"(blo), "r"(bhi), "r"(idesc), "r"(accum), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}

// 32 consecutive columns into r[OFF .. OFF + 31].
template <int OFF, int K>
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[K]) {
    static_assert(OFF + 32 <= K, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[OFF + 0]), "=r"(r[OFF + 1]), "=r"(r[OFF + 2]), "=r"(r[OFF + 3]), "=r"(r[OFF + 4]), "=r"(r[OFF + 5]),
          "=r"(r[OFF + 6]), "=r"(r[OFF + 7]), "=r"(r[OFF + 8]), "=r"(r[OFF + 9]), "=r"(r[OFF + 10]),
          "=r"(r[OFF + 11]), "=r"(r[OFF + 12]), "=r"(r[OFF + 13]), "=r"(r[OFF + 14]), "=r"(r[OFF + 15]),
          "=r"(r[OFF + 16]), "=r"(r[OFF + 17]), "=r"(r[OFF + 18]), "=r"(r[OFF + 19]), "=r"(r[OFF + 20]),
          "=r"(r[OFF + 21]), "=r"(r[OFF + 22]), "=r"(r[OFF + 23]), "=r"(r[OFF + 24]), "=r"(r[OFF + 25]),
          "=r"(r[OFF + 26]), "=r"(r[OFF + 27]), "=r"(r[OFF + 28]), "=r"(r[OFF + 29]), "=r"(r[OFF + 30]),
          "=r"(r[OFF + 31])
        : "r"(taddr));
}

// Registers per thread of this warpgroup, raised or lowered to N; the sum over
// the block's warpgroups stays within what it was launched with.
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

}  // namespace sm100
}  // namespace dcp
