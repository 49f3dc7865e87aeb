// attend_tc.cuh -- the 5th-generation tensor core's instructions as the attention
// kernels use them.
#pragma once

#include "attend_common.cuh"

namespace lbv {
namespace att {

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&d)[32])
{
    uint32_t* r = reinterpret_cast<uint32_t*>(d);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&d)[16])
{
    uint32_t* r = reinterpret_cast<uint32_t*>(d);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};\n" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
        "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Four steps of 16 of the contracted dimension, D (+)= A B, issued by one elected
// lane of a converged warp: their operands stay in uniform registers that way (a
// single thread in a branch of its own took 85 cycles an MMA to issue them).
// `add` 0: the first step overwrites D.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.b32 p, %10, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, 1;\n}\n" ::"r"(d), "l"(a), "l"(a + 2),
        "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc), "r"(add)
        : "memory");
}

// The same with A (P) in tensor memory and B (V) with its rows along the
// contracted dimension: 8 columns of A and 16 rows of B a step.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.b32 p, %10, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, 1;\n}\n" ::"r"(d), "r"(a),
        "r"(a + 8), "r"(a + 16), "r"(a + 24), "l"(b), "l"(b + 128), "l"(b + 256), "l"(b + 384),
        "r"(idesc), "r"(add)
        : "memory");
}

// Arrives on `bar` once every MMA the elected lane has issued is complete.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor in 128-byte-swizzled rows: 8-row groups 1024
// bytes apart; for an operand whose rows run along the contracted dimension (V),
// `lead` bytes between its 64-element column groups.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, fp32 sums, M = 128; bit 16: B is N-major.
template <int DT>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_n_major)
{
    return (1u << 4) | ((uint32_t)(DT == LBV_BF16) << 7) | ((uint32_t)(DT == LBV_BF16) << 10) |
           ((uint32_t)b_n_major << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;\n"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

}  // namespace att
}  // namespace lbv
