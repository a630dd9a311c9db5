// lora.cu — the low-rank adapters' share of a linear: h = scale_a * (x @ A_a^T) for each row's adapter a, then
// out = y + h @ B_a^T, with y the shared projection in fp32.
//
// The simple form: a warp for each inner value, a thread for each output.
#include <cuda_runtime.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

// h[t][r], 0 for a row without an adapter.
__global__ void __launch_bounds__(256) lora_inner_kernel(const LoraArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= (long long)a.M * a.R) return;
    const int t = (int)(i / a.R), r = (int)(i - (long long)t * a.R), id = a.ids[t];
    float sum = 0.0f;
    if ((unsigned)id < (unsigned)a.L) {
        const uint16_t *x = static_cast<const uint16_t *>(a.x) + (size_t)t * a.K;
        const uint16_t *w = static_cast<const uint16_t *>(a.a) + ((size_t)id * a.R + r) * a.K;
        for (int k = 2 * lane; k < a.K; k += 64)
            sum = fma2_bf16(*reinterpret_cast<const uint32_t *>(x + k), *reinterpret_cast<const uint32_t *>(w + k), sum);
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (a.scale) sum *= a.scale[id];
    }
    if (lane == 0) a.h[i] = sum;
}

__global__ void __launch_bounds__(256) lora_outer_kernel(const LoraArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)a.M * a.N) return;
    const int t = (int)(i / a.N), n = (int)(i - (long long)t * a.N), id = a.ids[t];
    float sum = a.y[i];
    if ((unsigned)id < (unsigned)a.L) {
        const uint16_t *b = static_cast<const uint16_t *>(a.b) + ((size_t)id * a.N + n) * a.R;
        const float *h = a.h + (size_t)t * a.R;
        float d = 0.0f;
        for (int r = 0; r < a.R; ++r) d = fmaf(h[r], bf16_to_f32(b[r]), d);
        sum += d;
    }
    static_cast<uint16_t *>(a.out)[i] = f32_to_bf16(sum);
}

int launch(void (*f)(const LoraArgs), long long blocks, const LoraArgs &a, uint32_t flags, void *stream) {
    if (blocks > 0x7FFFFFFFll) return (int)cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, f, a);
}

}  // namespace

int launch_lora_inner(const LoraArgs &a, uint32_t flags, void *stream) {
    return launch(lora_inner_kernel, ((long long)a.M * a.R + 7) / 8, a, flags, stream);
}

int launch_lora_outer(const LoraArgs &a, uint32_t flags, void *stream) {
    return launch(lora_outer_kernel, ((long long)a.M * a.N + 255) / 256, a, flags, stream);
}

}  // namespace bf16l
