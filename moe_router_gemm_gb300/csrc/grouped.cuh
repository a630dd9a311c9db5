// grouped.cuh — device helpers of the kernels whose weight depends on the row: TMA loads for a CTA pair from a stack of
// matrices, and copies of rows given by index.
#pragma once

#include "common.cuh"

namespace bf16l {

// As tma_load_2d_pair, from a stack of matrices: c0 innermost (K), c1 row, c2 half, c3 matrix.
__device__ __forceinline__ void tma_load_4d_pair(void *dst, const CUtensorMap *map, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// ... c0 innermost (K), c1 row of a block, c2 half, c3 block, c4 matrix.
__device__ __forceinline__ void tma_load_5d_pair(void *dst, const CUtensorMap *map, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(c4)
        : "memory");
}

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Sixteen bytes to shared memory, asynchronously: those from `bytes` (0 or 16) on are zero and not read.
__device__ __forceinline__ void cp_async_16(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// One arrival on an mbarrier of this CTA (of those that it was set up for) when this thread's copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Shared-memory matrix descriptor of a K-major bf16 tile of 16 columns (rows of 32 bytes, groups of eight of 256) in
// TMA's 32-byte swizzle; fields as smem_desc_sw128, swizzle mode 6.
__device__ __forceinline__ uint64_t smem_desc_sw32(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(256 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)6 << 61;
}

// As mma_bf16_pair, the operands given by the low words of their descriptors (smem_desc_sw128's high word is a constant),
// so that a step along K is one 32-bit addition.
__device__ __forceinline__ void mma_bf16_pair_sw128(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc,
                                                    uint32_t accumulate) {
    constexpr uint32_t kHigh = (uint32_t)((1024 >> 4) | 1 << 14 | 2u << 29);
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "n"(kHigh)
        : "memory");
}

// Two pair MMAs that add to D in the lanes (rows) alone whose bit of `off` is clear (words 0-3 the even CTA's, 4-7 the
// odd's): A0 B^T and A1 B^T, the A operands given by their descriptors' low words (128-byte swizzle).
__device__ __forceinline__ void mma_bf16_pair_lanes2(uint32_t d_tmem, uint32_t alo0, uint32_t alo1, uint64_t bdesc,
                                                     uint32_t idesc, const uint32_t (&off)[8]) {
    constexpr uint32_t kHigh = (uint32_t)((1024 >> 4) | 1 << 14 | 2u << 29);
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, c;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "mov.b64 a, {%1, %13};\n\t"
        "mov.b64 c, {%2, %13};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, %3, %4, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], c, %3, %4, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n\t}"
        ::"r"(d_tmem), "r"(alo0), "r"(alo1), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]),
        "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7]), "n"(kHigh)
        : "memory");
}

// g / (1 + exp(-g)), within 2^-20 of it: exp(-g) = 2^t (1 + r ln 2) with t + r = -g log2(e), t rounded and r what the rounding
// left and the part of log2(e) past 24 bits; a reciprocal and a product for the quotient.  The reciprocal is of a quarter of
// 1 + exp(-g), since below 2^-126 it would be 0, and of g's quarter the product.  From where exp(-g) overflows (g = -88.73) on
// the quotient is -0, and NaN for g = -infinity, as both are by a division in fp32.
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float t = -g * kLog2e;
    const float r = fmaf(-g, kLog2e, -t) - g * kLog2eLow;
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    if (fabsf(t) < 128.0f) e = fmaf(e * r, kLn2, e);  // (2^t finite, r small)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fmaf(0.25f, e, 0.25f)));
    return 0.25f * g * q;
}

// v as the sum of two bf16 values of its own sign: v cut off after eight bits, and the rounded rest, together off by at most
// 2^-16 of it, or 2^-132.  Products of both with an infinity then make the infinity that v's makes.  (With the first one
// rounded they are off by at most 2^-17, but a rest of the other sign, or none, makes NaN there: so none is 0 but for v = 0.)
__device__ __forceinline__ void two_bf16(float v, uint32_t &high, uint32_t &low) {
    const uint32_t bits = __float_as_uint(v) >> 16, sign = bits & 0x8000u, least = v != 0.0f;  // (2^-133)
    high = isnan(v) ? 0x7FFFu : max(bits & 0x7FFFu, least);
    low = isfinite(v) ? f32_to_bf16(fmaxf(fabsf(v) - bf16_to_f32((uint16_t)high), 0.0f)) : 0u;
    low = max(low, least) | sign;
    high |= sign;
}

// Host: a tensor map of a stack of bf16 matrices [planes][halves][rows][cols], dense, with a box of box_cols x box_rows x
// box_halves x 1 elements, in the swizzle of box_cols' bytes (128 or 32).  Defined in api.cu; a CUresult (0 on success).
int make_tmap_bf16_stack(CUtensorMap *map, const void *base, uint64_t planes, uint64_t halves, uint64_t rows, uint64_t cols,
                         uint32_t box_halves, uint32_t box_rows, uint32_t box_cols);
// The same with the rows in blocks of block_rows (a divisor of rows): a box is box_blocks blocks of every half, in shared
// memory block by block, a block's halves one after the other.
int make_tmap_bf16_blocks(CUtensorMap *map, const void *base, uint64_t planes, uint64_t halves, uint64_t rows, uint64_t cols,
                          uint32_t block_rows, uint32_t box_blocks, uint32_t box_cols);

}  // namespace bf16l
