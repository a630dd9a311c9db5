// lora.cu — the low-rank adapters' share of a linear for few rows: h = scale_a * (x @ A_a^T) for each row's adapter a, then
// out = y + h @ B_a^T, with y the shared projection in fp32, by the dense linear's own kernels between the two.
//
// Both kernels stand for little work (131 KB of an adapter of rank 16 and 4096 columns each way) and much latency, so each
// spreads over as many SMs as it can: the inner one a row's K over up to eight blocks, whose sums the outer one
// adds, in order, when it reads them, and four ranks a warp.  The inner one also asks L2 for B_a, which the outer one reads when the projection
// is done.
#include <cuda_runtime.h>

#include "grouped.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr int kInnerWarps = 4, kRanks = 4;  // ranks that a warp sums at a time
constexpr int kOuterThreads = 128;

// A warp sums kRanks ranks of a row over a part of K.
__global__ void __launch_bounds__(32 * kInnerWarps) lora_inner_kernel(const LoraArgs a) {
    const int splits = (int)gridDim.y;
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, s = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = __ldg(a.ids + t);
    if ((unsigned)id >= (unsigned)a.L) return;  // (its inner values are not read)
    if (threadIdx.x == 0 && blockIdx.z == 0) {  // this block's part of B's rows
        const int n0 = (int)((long long)a.N * s / splits), n1 = (int)((long long)a.N * (s + 1) / splits);
        const uint16_t *b = static_cast<const uint16_t *>(a.b) + ((size_t)id * a.N + n0) * a.R;
        const long long bytes = (long long)(n1 - n0) * a.R * 2;
        prefetch_l2(b, (uint32_t)(bytes < (1 << 20) ? bytes : 1 << 20));
    }
    const int r0 = kRanks * (kInnerWarps * (int)blockIdx.z + warp);
    if (r0 >= a.R) return;  // (R % 8 == 0)
    const int each = ((a.K + splits - 1) / splits + 255) / 256 * 256, k0 = s * each, k1 = min(k0 + each, a.K);
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + (size_t)t * a.K;
    const uint16_t *w = static_cast<const uint16_t *>(a.a) + ((size_t)id * a.R + r0) * a.K;
    float sum[kRanks] = {};
#pragma unroll 4
    for (int k = k0 + 8 * lane; k < k1; k += 256) {  // (K % 8 == 0)
        const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(x + k));
        uint4 wv[kRanks];
#pragma unroll
        for (int r = 0; r < kRanks; ++r) wv[r] = __ldg(reinterpret_cast<const uint4 *>(w + (size_t)r * a.K + k));
#pragma unroll
        for (int r = 0; r < kRanks; ++r) {
            sum[r] = fma2_bf16(xv.x, wv[r].x, sum[r]);
            sum[r] = fma2_bf16(xv.y, wv[r].y, sum[r]);
            sum[r] = fma2_bf16(xv.z, wv[r].z, sum[r]);
            sum[r] = fma2_bf16(xv.w, wv[r].w, sum[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < kRanks; ++r) {
#pragma unroll
        for (int d = 16; d; d >>= 1) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], d);
    }
    if (lane < kRanks) {
        float v = sum[0];
#pragma unroll
        for (int r = 1; r < kRanks; ++r) v = lane == r ? sum[r] : v;
        if (a.scale) v *= __ldg(a.scale + id);
        if (a.splits) {
            static_cast<float *>(a.h)[((size_t)s * a.M + t) * a.R + r0 + lane] = v;
        } else {
            uint32_t high, low;
            two_bf16(v, high, low);
            uint16_t *h = static_cast<uint16_t *>(a.h) + (size_t)t * 2 * a.R + r0 + lane;
            h[0] = (uint16_t)high;
            h[a.R] = (uint16_t)low;
        }
    }
}

// One output a thread: its B row is R consecutive values.
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(const LoraArgs a) {
    __shared__ float h[kLoraMaxRank];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, id = __ldg(a.ids + t);
    const bool has = (unsigned)id < (unsigned)a.L;
    if (has && (int)threadIdx.x < a.R) {
        float v = 0.0f;
        const uint16_t *two = static_cast<const uint16_t *>(a.h) + (size_t)t * 2 * a.R + threadIdx.x;
        if (!a.splits) v = bf16_to_f32(two[0]) + bf16_to_f32(two[a.R]);
        for (int s = 0; s < a.splits; ++s) v += static_cast<const float *>(a.h)[((size_t)s * a.M + t) * a.R + threadIdx.x];
        h[threadIdx.x] = v;
    }
    __syncthreads();
    for (long long n = (long long)blockIdx.y * kOuterThreads + threadIdx.x; n < a.N; n += (long long)gridDim.y * kOuterThreads) {
        const size_t at = (size_t)t * a.N + n;
        float sum = a.y[at];
        if (has) {
            const uint4 *b = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.b) + ((size_t)id * a.N + n) * a.R);
            float d = 0.0f;
#pragma unroll 4
            for (int i = 0; i < a.R / 8; ++i) {
                const uint4 v = __ldg(b + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d = fmaf(h[8 * i + 2 * j], bf16_lo(w[j]), d);
                    d = fmaf(h[8 * i + 2 * j + 1], bf16_hi(w[j]), d);
                }
            }
            sum += d;
        }
        static_cast<uint16_t *>(a.out)[at] = f32_to_bf16(sum);
    }
}

int launch(void (*f)(const LoraArgs), dim3 grid, int threads, const LoraArgs &a, uint32_t flags, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, f, a);
}

}  // namespace

// None below 512 elements.
int lora_splits(int K) {
    const int s = K / 512 > 1 ? K / 512 : 1;
    return s < 8 ? s : 8;
}

int launch_lora_inner(const LoraArgs &a, uint32_t flags, void *stream) {
    const int ranks = kRanks * kInnerWarps;
    const dim3 grid((unsigned)a.M, (unsigned)(a.splits ? a.splits : 1), (unsigned)((a.R + ranks - 1) / ranks));
    return launch(lora_inner_kernel, grid, 32 * kInnerWarps, a, flags, stream);
}

int launch_lora_outer(const LoraArgs &a, uint32_t flags, void *stream) {
    const int blocks = (a.N + kOuterThreads - 1) / kOuterThreads;
    const dim3 grid((unsigned)a.M, (unsigned)(blocks < 65535 ? blocks : 65535));
    return launch(lora_outer_kernel, grid, kOuterThreads, a, flags, stream);
}

}  // namespace bf16l
