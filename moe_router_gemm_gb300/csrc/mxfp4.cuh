// mxfp4.cuh — device helpers of the 4-bit microscaled format: 32 elements along
// K share one E8M0 scale byte e (2^(e - 127), 255 = NaN), the elements are e2m1
// codes (sign, 2 exponent bits of bias 1, 1 mantissa bit), two to a byte.
#pragma once

#include "common.cuh"

namespace bf16l {

// 2^(e - 127) as fp32: normal for e in 1..254, the subnormal 2^-127 for 0, NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t e) {
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}

// Eight fp32 values -> eight e2m1 codes in one word, v[0] in the low four bits:
// round to nearest even, saturating at +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The block's scale exponent s = max(floor(log2 amax) - top, -127) from amax's
// bits (fp32, finite or infinite, sign clear): the exponent field is floor(log2)
// + 127, and 0 (zero and subnormals) lies below the clamp.  top: the exponent of
// the element format's largest binade (2 for e2m1, 8 for e4m3).
__device__ __forceinline__ int mx_scale_exp(uint32_t amax_bits, int top) {
    const int s = (int)(amax_bits >> 23) - 127 - top;
    return s < -127 ? -127 : s;
}

// 2^-s for s in [-127, 126]: always a normal fp32 number.
__device__ __forceinline__ float exp2_neg(int s) { return __uint_as_float((uint32_t)(127 - s) << 23); }

// Quantise 8 consecutive bf16 values (one 16-byte vector) of a block that four
// neighbouring lanes (a quad) hold: the codes of this lane's 8 values, and the
// scale byte.  All four lanes of the quad must call it together.  Magnitudes
// compare as integers, so a NaN is the largest and shows in the maximum.
__device__ __forceinline__ uint32_t mxfp4_quant_vec(const uint4 &w, unsigned quad, uint32_t &scale_byte) {
    uint32_t m2 = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                           __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
    m2 = __vmaxu2(m2, __shfl_xor_sync(quad, m2, 1));
    m2 = __vmaxu2(m2, __shfl_xor_sync(quad, m2, 2));
    const uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
    const bool nan = amax > 0x7F80u;
    const int s = mx_scale_exp(amax << 16, 2);
    const float inv = exp2_neg(nan ? 0 : s);
    const float f[8] = {bf16_lo(w.x) * inv, bf16_hi(w.x) * inv, bf16_lo(w.y) * inv, bf16_hi(w.y) * inv,
                        bf16_lo(w.z) * inv, bf16_hi(w.z) * inv, bf16_lo(w.w) * inv, bf16_hi(w.w) * inv};
    scale_byte = nan ? 255u : (uint32_t)(s + 127);
    return nan ? 0u : e2m1x8(f);
}

// Instruction descriptor of the block-scaled e2m1 MMA (kind::mxf4): A and B e2m1
// (format 1 at bits 7-9 and 10-12), K-major, N>>3 at bit 17, scale format E8M0
// at bit 23, M>>4 at bit 24; the first of the two bytes of each 32-bit scale word
// to use (0 or 2) at bits 4-5 for B and 29-30 for A.  D is fp32.
__host__ __device__ constexpr uint32_t idesc_mxf4_f32(int mma_m, int mma_n, int sf_id) {
    return (1u << 7) | (1u << 10) | ((uint32_t)sf_id << 4) | ((uint32_t)(mma_n >> 3) << 17) | (1u << 23) |
           ((uint32_t)(mma_m >> 4) << 24) | ((uint32_t)sf_id << 29);
}

// One block-scaled e2m1 MMA, K = 64 codes (two scale blocks, 32 bytes of a row):
// D[tmem] (+)= (A * sA) (B * sB)^T.  Scale words in TMEM as for mma_mxf8, at
// columns that are multiples of 8.
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// The same by a CTA pair (M = 256: each CTA's own 128 A rows and accumulator rows, each holds
// half of the B rows), issued by one thread of the even CTA.  Each CTA's TMEM holds the scales
// of its own A rows and of all B rows, at the same columns in both.
__device__ __forceinline__ void mma_mxf4_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
        : "memory");
}

// Asks for the 16-byte block at p (16-byte aligned) in shared memory at `to`, of which only the part inside [lo, hi) is
// read.  The array's first block, where it starts within one, is there on return.
__device__ __forceinline__ void copy_block(uint4 *to, const uint8_t *p, const uint8_t *lo, const uint8_t *hi) {
    if (p >= lo) {
        const long long left = hi - p;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(p),
                     "r"(left < 16 ? (int)left : 16)
                     : "memory");
        return;
    }
#pragma unroll 1
    for (int i = (int)(lo - p); i < 16 && p + i < hi; ++i) reinterpret_cast<uint8_t *>(to)[i] = __ldg(p + i);
}
// Sixteen scale bytes, 1.0 from byte n on.
__device__ __forceinline__ uint4 scales_until(const uint4 &q, int n) {
    if (n >= 16) return q;
    uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int left = n - 4 * j;  // valid bytes of this word
        const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        w[j] = (w[j] & keep) | (0x7F7F7F7Fu & ~keep);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's newest N groups of copies are complete.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sixteen bytes from byte m (below 16) of two neighbouring blocks on.
__device__ __forceinline__ uint4 shift_blocks(const uint4 &a, const uint4 &b, int m) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t[7], v[5];  // words (m / 4) & 1 on, then m / 4 on
#pragma unroll
    for (int k = 0; k < 7; ++k) t[k] = m & 4 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) v[k] = m & 8 ? t[k + 2] : t[k];
    const int s = 8 * (m & 3);
    return make_uint4(__funnelshift_r(v[0], v[1], s), __funnelshift_r(v[1], v[2], s), __funnelshift_r(v[2], v[3], s),
                      __funnelshift_r(v[3], v[4], s));
}

// Arrive on an mbarrier of a CTA of the cluster, ordering this thread's earlier
// accesses for its own CTA only.  Enough where what the arrival announces is read
// through the async proxy (a fence.proxy.async came before it) or by tcgen05: a
// release at cluster scope, and the acquire that goes with it, cost about a
// microsecond a chunk here.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Barrier `id` for `threads` threads of the CTA (whole warps).
__device__ __forceinline__ void named_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// TMA store of a tile from shared memory (c0 innermost, c0 and c1 not negative), a
// bulk group of its own; what lies past the matrix is not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
// This thread's bulk stores have read their shared memory / are complete.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace bf16l
