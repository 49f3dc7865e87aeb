// kv4.cuh -- where a cache of 4 bits holds what, and its values.
//
// A page is [heads][chunks of C = min(page_size, 64) slots]; a chunk is codes
// [K, V][D / 64][C][32 bytes], then scales [K, V][D / 64][C] of (scale, bias).  So what a
// kernel takes of a head's slots at once, keys and values, is one stretch of memory
// (9,216 bytes for 64 slots of 128 elements), and a lane's 8 or 16 bytes of codes
// come from rows of 32 bytes, four of which fill the banks of shared memory.  In a
// word of 8 codes the even elements are in the low half and the odd ones in the
// high half, so that a mask leaves two neighbours where a pair of 16-bit values has them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "step_internal.h"

namespace lbv {
namespace kv4 {

constexpr int kSlotBytes = 72;        // of 64 elements of a key and a value: 2 (32 + 4)

__host__ __device__ __forceinline__ int chunk_shift(const KvView& kv)
{
    return kv.page_shift < 6 ? kv.page_shift : 6;
}

// Bytes of one slot of a head.
__host__ __device__ __forceinline__ int slot_bytes(int dim)
{
    return dim / 64 * kSlotBytes;
}

__host__ __device__ __forceinline__ int64_t page_bytes(const KvView& kv)
{
    return (int64_t)kv.heads * slot_bytes(kv.dim) << kv.page_shift;
}

#ifdef __CUDACC__
// The chunk that holds `slot` of a page.
__device__ __forceinline__ uint8_t* chunk(const KvView& kv, int page, int head, int slot)
{
    const int cs = chunk_shift(kv), per = slot_bytes(kv.dim);
    return kv.packed + ((int64_t)page * kv.heads + head) * ((int64_t)per << kv.page_shift) +
           (int64_t)(slot >> cs) * (per << cs);
}

// Offsets in a chunk of slot s: codes (32 bytes) and (scale, bias) of plane
// which * D / 64 + part.
__device__ __forceinline__ int codes_at(int plane, int s, int cs)
{
    return ((plane << cs) + s) * 32;
}

__device__ __forceinline__ int scale_at(int planes, int plane, int s, int cs)
{
    return (planes * 32 << cs) + ((plane << cs) + s) * 4;
}

// (x & mask) | bits, in one instruction.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(r) : "r"(x), "n"(MASK), "r"(bits));
    return r;
}

// Constants of expand() that an instruction cannot hold beside another: kept in registers, by a
// kernel that makes them once.  (Left to the compiler they were made anew for every word.)
struct Constants {
    uint32_t bits, many;
};

template <int DT>
__device__ __forceinline__ Constants constants()
{
    Constants c;
    asm volatile("mov.b32 %0, %1;\n" : "=r"(c.bits) : "n"(DT == LBV_F16 ? 0x64006400 : 0x43004300));
    asm volatile("mov.b32 %0, %1;\n" : "=r"(c.many) : "n"(0xD400D400));      // -64, -64
    return c;
}

// The pairs at the four places of a word w: out[i] = code * scale + bias, rounded once,
// of the codes in bits 4 i and 4 i + 16 on (of one slot's word elements 2 i and 2 i + 1).
//
// A code goes to the low mantissa bits of 1024 (fp16) or 128 (bf16) by one logical
// instruction; the subtraction of that number is exact.  (fp16 has room for the code four bits
// up, too: 1024 + 16 c, so a shift serves two pairs.)
template <int DT>
__device__ __forceinline__ void expand(uint32_t w, uint32_t scale2, uint32_t bias2, const Constants& k,
                                       uint32_t (&out)[4])
{
    if constexpr (DT == LBV_F16) {
        const __half2 s = reinterpret_cast<const __half2&>(scale2), b = reinterpret_cast<const __half2&>(bias2);
        const __half2 many = reinterpret_cast<const __half2&>(k.many);
        const __half2 one = __float2half2_rn(-1024.f), sixteenth = __float2half2_rn(0.0625f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = w >> (8 * i);
            const uint32_t lo = pick<0x000F000Fu>(x, k.bits), hi = pick<0x00F000F0u>(x, k.bits);
            const __half2 a = __hadd2(reinterpret_cast<const __half2&>(lo), one);
            const __half2 c = __hfma2(reinterpret_cast<const __half2&>(hi), sixteenth, many);
            reinterpret_cast<__half2&>(out[2 * i]) = __hfma2(a, s, b);
            reinterpret_cast<__half2&>(out[2 * i + 1]) = __hfma2(c, s, b);
        }
    } else {
        const __nv_bfloat162 s = reinterpret_cast<const __nv_bfloat162&>(scale2),
                             b = reinterpret_cast<const __nv_bfloat162&>(bias2);
        const __nv_bfloat162 one = __float2bfloat162_rn(-128.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = pick<0x000F000Fu>(w >> (4 * i), k.bits);
            const __nv_bfloat162 a = __hadd2(reinterpret_cast<const __nv_bfloat162&>(lo), one);
            reinterpret_cast<__nv_bfloat162&>(out[i]) = __hfma2(a, s, b);
        }
    }
}

// (scale, scale) and (bias, bias) of a stored pair.
__device__ __forceinline__ uint32_t both_scales(uint32_t sb)
{
    return __byte_perm(sb, sb, 0x1010);
}

__device__ __forceinline__ uint32_t both_biases(uint32_t sb)
{
    return __byte_perm(sb, sb, 0x3232);
}
#endif

}  // namespace kv4
}  // namespace lbv
