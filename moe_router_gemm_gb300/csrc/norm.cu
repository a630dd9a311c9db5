// norm.cu — root-mean-square norm of rows, with the residual's addition before
// it and an output in bf16 and / or in 8 or 4 bits with scales.
//
//     h = x  or  RNE_bf16(x + residual);  y = h / sqrt(mean(h^2) + eps) * weight
//
// One pass: a block holds its row in registers between the sum of squares and
// the output, so each input is read once and each output written once.  The sum
// runs in fp32: each thread over its own values in order, then a shuffle tree,
// then the warps in order, so it is the same from run to run.
//
//   * norm_vec_kernel: rows that start on 16-byte boundaries (H and ldx multiples
//     of 8): thread i holds the 8-value vectors i, i + threads, ...; four
//     neighbouring lanes hold a 32-element scale block.
//   * norm_any_kernel: any H, stride and alignment, one value per lane and step;
//     a warp's 32 lanes hold a scale block.  Reads the row twice (the second
//     time from L1 or L2).
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

struct NormArgs {
    const uint16_t *x;
    const uint16_t *residual;
    const uint16_t *weight;
    uint16_t *out;
    uint16_t *residual_out;
    uint8_t *codes;
    uint8_t *scales;
    const float *scale;
    long long rows, ldx;
    int H;
    float eps;
};

__device__ __forceinline__ uint16_t e4m3x2_sat(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Sum over the block, the same in every thread.  `red`: one float per warp.
__device__ __forceinline__ float block_sum(float v, float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (int)blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += red[w];
    __syncthreads();  // red is free again
    return s;
}

// Magnitude bits of a value for a block's maximum: NaN above infinity, so it shows.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

template <int QUANT, int V>
__global__ void __launch_bounds__(1024) norm_vec_kernel(const NormArgs a) {
    __shared__ float red[32];
    pdl_launch_dependents();
    pdl_wait();  // x, the residual, the weight and the scale may be written by the previous kernel
    const int nvec = a.H >> 3, nt = (int)blockDim.x;
    const float inv_scale = QUANT == BF16L_QUANT_FP8 ? 1.0f / __ldg(a.scale) : 0.0f;
    const unsigned quad = 0xFu << (threadIdx.x & 28u);
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + r * a.ldx);
        uint4 h[V];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = (int)threadIdx.x + j * nt;
            h[j] = i < nvec ? __ldg(xr + i) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (a.residual) {
            const uint4 *rr = reinterpret_cast<const uint4 *>(a.residual + r * a.H);
            uint4 q[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int i = (int)threadIdx.x + j * nt;
                q[j] = i < nvec ? rr[i] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[j].x = pack_bf16x2(bf16_lo(h[j].x) + bf16_lo(q[j].x), bf16_hi(h[j].x) + bf16_hi(q[j].x));
                h[j].y = pack_bf16x2(bf16_lo(h[j].y) + bf16_lo(q[j].y), bf16_hi(h[j].y) + bf16_hi(q[j].y));
                h[j].z = pack_bf16x2(bf16_lo(h[j].z) + bf16_lo(q[j].z), bf16_hi(h[j].z) + bf16_hi(q[j].z));
                h[j].w = pack_bf16x2(bf16_lo(h[j].w) + bf16_lo(q[j].w), bf16_hi(h[j].w) + bf16_hi(q[j].w));
                const int i = (int)threadIdx.x + j * nt;
                if (i < nvec) reinterpret_cast<uint4 *>(a.residual_out + r * a.H)[i] = h[j];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint32_t u[4] = {h[j].x, h[j].y, h[j].z, h[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ss = fmaf(bf16_lo(u[e]), bf16_lo(u[e]), ss);
                ss = fmaf(bf16_hi(u[e]), bf16_hi(u[e]), ss);
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red) / (float)a.H + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = (int)threadIdx.x + j * nt;
            if (i >= nvec) break;  // nvec % 4 == 0 for the MX formats: a quad leaves together
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(a.weight) + i);
            const uint32_t u[4] = {h[j].x, h[j].y, h[j].z, h[j].w}, g[4] = {w.x, w.y, w.z, w.w};
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[2 * e] = bf16_lo(u[e]) * rstd * bf16_lo(g[e]);
                y[2 * e + 1] = bf16_hi(u[e]) * rstd * bf16_hi(g[e]);
            }
            if (a.out) OutStore<uint16_t>::eight(a.out + r * a.H + 8 * (long long)i, y);
            if (QUANT == BF16L_QUANT_FP8) {
                uint16_t c[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = e4m3x2_sat(y[2 * e] * inv_scale, y[2 * e + 1] * inv_scale);
                reinterpret_cast<uint2 *>(a.codes + r * a.H)[i] =
                    make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16), (uint32_t)c[2] | ((uint32_t)c[3] << 16));
            } else if (QUANT != BF16L_QUANT_NONE) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, mag_bits(y[e]));
                m = max(m, __shfl_xor_sync(quad, m, 1));
                m = max(m, __shfl_xor_sync(quad, m, 2));
                const bool nan = m > 0x7F800000u;
                const int s = mx_scale_exp(m, QUANT == BF16L_QUANT_MXFP8 ? 8 : 2);
                const float inv = exp2_neg(nan ? 0 : s);
                if (QUANT == BF16L_QUANT_MXFP8) {
                    uint16_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = e4m3x2_sat(y[2 * e] * inv, y[2 * e + 1] * inv);
                    reinterpret_cast<uint2 *>(a.codes + r * a.H)[i] =
                        make_uint2((uint32_t)c[0] | ((uint32_t)c[1] << 16), (uint32_t)c[2] | ((uint32_t)c[3] << 16));
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= inv;
                    reinterpret_cast<uint32_t *>(a.codes + r * (a.H >> 1))[i] = nan ? 0u : e2m1x8(y);
                }
                if ((threadIdx.x & 3) == 0) a.scales[r * (a.H >> 5) + (i >> 2)] = nan ? 255 : (uint8_t)(s + 127);
            }
        }
    }
}

template <int QUANT>
__global__ void __launch_bounds__(512) norm_any_kernel(const NormArgs a) {
    __shared__ float red[32];
    pdl_launch_dependents();
    pdl_wait();
    const int nt = (int)blockDim.x, lane = threadIdx.x & 31;
    const float inv_scale = QUANT == BF16L_QUANT_FP8 ? 1.0f / __ldg(a.scale) : 0.0f;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const uint16_t *xr = a.x + r * a.ldx;
        const uint16_t *hr = a.residual ? a.residual_out + r * a.H : xr;  // where h is read from the second time
        float ss = 0.0f;
        for (int i = (int)threadIdx.x; i < a.H; i += nt) {
            float h = bf16_to_f32(xr[i]);
            if (a.residual) {
                const uint16_t b = f32_to_bf16(h + bf16_to_f32(a.residual[r * a.H + i]));
                a.residual_out[r * a.H + i] = b;  // read back below by this same thread
                h = bf16_to_f32(b);
            }
            ss = fmaf(h, h, ss);
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red) / (float)a.H + a.eps);
        for (int i = (int)threadIdx.x; i < a.H; i += nt) {
            const float y = bf16_to_f32(hr[i]) * rstd * bf16_to_f32(__ldg(a.weight + i));
            if (a.out) a.out[r * a.H + i] = f32_to_bf16(y);
            if (QUANT == BF16L_QUANT_FP8) {
                a.codes[r * a.H + i] = (uint8_t)(e4m3x2_sat(y * inv_scale, 0.0f) & 0xFFu);
            } else if (QUANT != BF16L_QUANT_NONE) {  // H % 32 == 0: a warp's lanes are one block, together in the loop
                uint32_t m = mag_bits(y);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const bool nan = m > 0x7F800000u;
                const int s = mx_scale_exp(m, QUANT == BF16L_QUANT_MXFP8 ? 8 : 2);
                const float v = y * exp2_neg(nan ? 0 : s);
                if (QUANT == BF16L_QUANT_MXFP8) {
                    a.codes[r * a.H + i] = (uint8_t)(e4m3x2_sat(v, 0.0f) & 0xFFu);
                } else {
                    const float w[8] = {v, __shfl_down_sync(0xFFFFFFFFu, v, 1), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    const uint32_t c = nan ? 0u : e2m1x8(w);
                    if ((lane & 1) == 0) a.codes[r * (a.H >> 1) + (i >> 1)] = (uint8_t)c;
                }
                if (lane == 0) a.scales[r * (a.H >> 5) + (i >> 5)] = nan ? 255 : (uint8_t)(s + 127);
            }
        }
    }
}

using NormFn = void (*)(const NormArgs);

template <int QUANT>
NormFn pick_vec(int v) {
    return v == 1 ? norm_vec_kernel<QUANT, 1> : v == 2 ? norm_vec_kernel<QUANT, 2> : norm_vec_kernel<QUANT, 4>;
}

}  // namespace

int launch_rmsnorm(const void *x, int64_t ldx, const void *residual, const void *weight, void *out, void *residual_out,
                   void *codes, void *scales, const float *scale, int64_t rows, int H, float eps, int quant,
                   int num_sms, uint32_t flags, void *stream) {
    NormArgs a = {static_cast<const uint16_t *>(x),
                  static_cast<const uint16_t *>(residual),
                  static_cast<const uint16_t *>(weight),
                  static_cast<uint16_t *>(out),
                  static_cast<uint16_t *>(residual_out),
                  static_cast<uint8_t *>(codes),
                  static_cast<uint8_t *>(scales),
                  scale,
                  rows,
                  ldx,
                  H,
                  eps};
    const bool vec = H % 8 == 0 && ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && H <= 8 * 4 * 1024;
    int threads;
    NormFn fn;
    if (vec) {
        const int nvec = H / 8;
        const int v = nvec <= 256 ? 1 : nvec <= 2048 ? 2 : 4;
        threads = ((nvec + v - 1) / v + 31) / 32 * 32;
        fn = quant == BF16L_QUANT_NONE    ? pick_vec<BF16L_QUANT_NONE>(v)
             : quant == BF16L_QUANT_FP8   ? pick_vec<BF16L_QUANT_FP8>(v)
             : quant == BF16L_QUANT_MXFP8 ? pick_vec<BF16L_QUANT_MXFP8>(v)
                                          : pick_vec<BF16L_QUANT_MXFP4>(v);
    } else {
        threads = H <= 512 ? (H + 31) / 32 * 32 : 512;
        fn = quant == BF16L_QUANT_NONE    ? norm_any_kernel<BF16L_QUANT_NONE>
             : quant == BF16L_QUANT_FP8   ? norm_any_kernel<BF16L_QUANT_FP8>
             : quant == BF16L_QUANT_MXFP8 ? norm_any_kernel<BF16L_QUANT_MXFP8>
                                          : norm_any_kernel<BF16L_QUANT_MXFP4>;
    }
    const long long cap = (long long)num_sms * (2048 / threads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows < cap ? rows : cap));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace bf16l
