// tcgen05.cuh -- sm_100a tensor-core helpers: tensor memory, shared-memory
// operand descriptors, the f16/bf16 matrix instruction and tiled TMA loads.
// One CTA only (cta_group::1), no multicast.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "tma.cuh"

namespace ssm {

// ---------------------------------------------------------- tensor memory --
// (a whole warp allocates and frees)
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(columns)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: register i of a lane is column i of its row.
// The wait is part of the statement, so nothing can use the registers before it.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
// Two stretches at once, with one wait (a load and its wait take some 160 cycles).
__device__ __forceinline__ void tmem_ld16x2(uint32_t at0, uint32_t at1, uint32_t (&r)[16], uint32_t (&q)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]),
            "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
        : "r"(at0), "r"(at1)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16x3(uint32_t at0, uint32_t at1, uint32_t at2, uint32_t (&r)[16], uint32_t (&q)[16],
                                            uint32_t (&o)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%48];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%49];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%50];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]),
            "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]),
          "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
            "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
        : "r"(at0), "r"(at1), "r"(at2)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// ------------------------------------------------------------- operands --
// A shared-memory tile here is rows of 128 bytes (64 elements) in the 128-byte
// swizzle that TMA writes: 16-byte piece i of row r lies at r * 128 + ((i ^ (r & 7)) * 16);
// groups of 8 rows are 1024 bytes apart.  The same tile serves with its rows as
// the product's depth (transposed operand: 64 consecutive elements of M or N per
// row, the next 64 `block` bytes away) or with its row elements as the depth.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t block) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((block >> 4) & 0x3fff) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// The matrix instructions and their commit are called by a whole converged warp
// and issued by one elected lane of it: with control flow and operands uniform
// over the warp, descriptors stay in uniform registers (issued from a branch of
// one lane, each instruction cost some 90 cycles of moves).
//
// f32 accumulator; type: 0 = f16, 1 = bf16 for both operands
__device__ __forceinline__ constexpr uint32_t mma_desc(uint32_t type, bool trans_a, bool trans_b, uint32_t m, uint32_t n) {
    return 1u << 4 | type << 7 | type << 10 | (trans_a ? 1u : 0u) << 15 | (trans_b ? 1u : 0u) << 16 | (n >> 3) << 17 |
           (m >> 4) << 24;
}
//
// A product over a depth of 128, eight instructions of 16 (one statement each, so
// that the elected lane is found once and the code stays small): operand
// descriptors advance by A1, A2 (B1, B2) in turn, 4 steps of the first, then the second -- for
// tiles whose row elements are the depth, 2 (32 bytes) three times, then on to the
// next tile.
#define SSM_MMA8_STEP(A)                                                            \
    "@e tcgen05.mma.cta_group::1.kind::f16 [%0], " A ", b, %3, 1;\n\t"
template <int A_STEP, int A_JUMP, int B_STEP, int B_JUMP>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc) {
    asm volatile(
        "{\n\t.reg .pred e, z;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 z, 0, 0;\n\t"
        "mov.b64 a, %1;\n\tmov.b64 b, %2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, z;\n\t"
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %5;\n\tadd.u64 b, b, %7;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "add.u64 a, a, %4;\n\tadd.u64 b, b, %6;\n\t" SSM_MMA8_STEP("a")
        "}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "n"(A_STEP), "n"(A_JUMP), "n"(B_STEP), "n"(B_JUMP)
        : "memory");
}
#undef SSM_MMA8_STEP
// left operand in tensor memory: two 16-bit depth elements per column
template <int B_STEP>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc) {
    asm volatile(
        "{\n\t.reg .pred e, z;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 z, 0, 0;\n\t"
        "mov.b32 a, %1;\n\tmov.b64 b, %2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, z;\n\t"
#define SSM_MMA8_STEP "add.u32 a, a, 8;\n\tadd.u64 b, b, %4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, 1;\n\t"
        SSM_MMA8_STEP SSM_MMA8_STEP SSM_MMA8_STEP SSM_MMA8_STEP SSM_MMA8_STEP SSM_MMA8_STEP SSM_MMA8_STEP
#undef SSM_MMA8_STEP
        "}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "n"(B_STEP)
        : "memory");
}
// the barrier is arrived at when every matrix instruction issued so far is done
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// box of a rank-4 tensor map into this CTA's shared memory; x times the element
// size is a multiple of 16 bytes
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

}  // namespace ssm
