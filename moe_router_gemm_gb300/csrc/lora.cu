// lora.cu — the low-rank adapters' share of a linear for few rows: h = scale_a * (x @ A_a^T) for each row's adapter a, then
// out = y + h @ B_a^T, with y the shared projection in fp32, by the dense linear's own kernels between the two.
//
// Both kernels stand for little work (131 KB of an adapter of rank 16 and 4096 columns each way) and much latency, so each
// spreads over as many SMs as it can: the inner one takes four ranks of a row a block and its K over up to eight blocks,
// whose sums the outer one adds, in order, when it reads them.  The inner one also asks L2 for B_a, which the outer one reads when the projection
// is done.
#include <cuda_runtime.h>

#include "grouped.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr int kInnerWarps = 4, kRanks = 4;  // ranks of a block
constexpr int kOuterThreads = 128;

// A block sums kRanks ranks of a row over a part of K, its warps taking 256 elements in turn.
__global__ void __launch_bounds__(32 * kInnerWarps) lora_inner_kernel(const LoraArgs a) {
    __shared__ float part[kInnerWarps][kRanks];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, s = blockIdx.y, splits = (int)gridDim.y, r0 = kRanks * (int)blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = __ldg(a.ids + t);
    if ((unsigned)id >= (unsigned)a.L) return;  // (its inner values are not read)
    if (threadIdx.x == 0 && a.splits) {  // this block's part of B's rows, for the outer kernel
        const int blocks = splits * (int)gridDim.z, i = s + splits * (int)blockIdx.z;
        const int n0 = (int)((long long)a.N * i / blocks), n1 = (int)((long long)a.N * (i + 1) / blocks);
        const uint16_t *b = static_cast<const uint16_t *>(a.b) + ((size_t)id * a.N + n0) * a.R;
        const long long bytes = (long long)(n1 - n0) * a.R * 2;
        prefetch_l2(b, (uint32_t)(bytes < (1 << 20) ? bytes : 1 << 20));
    }
    constexpr int kStep = 256 * kInnerWarps;
    const int each = ((a.K + splits - 1) / splits + kStep - 1) / kStep * kStep, k0 = s * each, k1 = min(k0 + each, a.K);
    const uint16_t *x = static_cast<const uint16_t *>(a.x) + (size_t)t * a.K;
    const uint16_t *w = static_cast<const uint16_t *>(a.a) + ((size_t)id * a.R + r0) * a.K;  // (R % 8 == 0)
    float sum[kRanks] = {};
#pragma unroll 4
    for (int k = k0 + 256 * warp + 8 * lane; k < k1; k += kStep) {  // (K % 8 == 0)
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
        if (lane == r) part[warp][r] = sum[r];
    }
    __syncthreads();
    if (threadIdx.x < kRanks) {
        const int r = threadIdx.x;
        float v = part[0][r];
#pragma unroll
        for (int i = 1; i < kInnerWarps; ++i) v += part[i][r];
        if (a.scale) v *= __ldg(a.scale + id);
        if (a.splits) {
            static_cast<float *>(a.h)[((size_t)s * a.M + t) * a.R + r0 + r] = v;
        } else {
            uint32_t high, low;
            two_bf16(v, high, low);
            uint16_t *h = static_cast<uint16_t *>(a.h) + (size_t)t * 2 * a.R + r0 + r;
            h[0] = (uint16_t)high;
            h[a.R] = (uint16_t)low;
        }
    }
}

// One output a thread: its B row is R consecutive values, the first kAhead vectors of which are on their way before the
// block has its h.
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(const LoraArgs a) {
    constexpr int kAhead = 4;
    __shared__ float h[kLoraMaxRank];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, id = __ldg(a.ids + t);
    const bool has = (unsigned)id < (unsigned)a.L;
    const uint16_t *B = static_cast<const uint16_t *>(a.b) + (has ? (size_t)id * a.N * a.R : 0);
    long long n = (long long)blockIdx.y * kOuterThreads + threadIdx.x;
    uint4 v[kAhead] = {};
    float y = 0.0f;
    auto load = [&]() {
        if (n >= a.N) return;
        y = a.y[(size_t)t * a.N + n];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (has && 8 * i < a.R) v[i] = __ldg(reinterpret_cast<const uint4 *>(B + n * a.R) + i);
    };
    load();
    if (has && (int)threadIdx.x < a.R) {
        float sum = 0.0f;
        const uint16_t *two = static_cast<const uint16_t *>(a.h) + (size_t)t * 2 * a.R + threadIdx.x;
        if (!a.splits) sum = bf16_to_f32(two[0]) + bf16_to_f32(two[a.R]);
#pragma unroll 8
        for (int s = 0; s < a.splits; ++s) sum += static_cast<const float *>(a.h)[((size_t)s * a.M + t) * a.R + threadIdx.x];
        h[threadIdx.x] = sum;
    }
    __syncthreads();
    while (n < a.N) {
        float d = 0.0f;
        auto add = [&](const uint4 &q, int i) {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d = fmaf(h[8 * i + 2 * j], bf16_lo(w[j]), d);
                d = fmaf(h[8 * i + 2 * j + 1], bf16_hi(w[j]), d);
            }
        };
        if (has) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (8 * i < a.R) add(v[i], i);
            for (int i = kAhead; i < a.R / 8; ++i) add(__ldg(reinterpret_cast<const uint4 *>(B + n * a.R) + i), i);
        }
        static_cast<uint16_t *>(a.out)[(size_t)t * a.N + n] = f32_to_bf16(y + d);
        n += (long long)gridDim.y * kOuterThreads;
        load();
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

// Blocks for each SM eight times over, none below a step of K.
int lora_splits(int M, int K, int R) {
    const long long blocks = (long long)M * (R / kRanks), want = (8 * kGb300Sms + blocks - 1) / blocks;
    const long long most = K / (256 * kInnerWarps) < 8 ? K / (256 * kInnerWarps) : 8, s = want < most ? want : most;
    return s < 1 ? 1 : (int)s;
}

int launch_lora_inner(const LoraArgs &a, uint32_t flags, void *stream) {
    const dim3 grid((unsigned)a.M, (unsigned)(a.splits ? a.splits : 1), (unsigned)(a.R / kRanks));
    return launch(lora_inner_kernel, grid, 32 * kInnerWarps, a, flags, stream);
}

int launch_lora_outer(const LoraArgs &a, uint32_t flags, void *stream) {
    const int blocks = (a.N + kOuterThreads - 1) / kOuterThreads;
    const dim3 grid((unsigned)a.M, (unsigned)(blocks < 65535 ? blocks : 65535));
    return launch(lora_outer_kernel, grid, kOuterThreads, a, flags, stream);
}

}  // namespace bf16l
