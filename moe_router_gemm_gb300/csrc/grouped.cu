// grouped.cu — out[p] = x[row of p] @ W[e]^T (+ bias[e]) for the rows p of each group e, their numbers known on the
// device alone; with SwiGLU, W[e] holds N gate rows and then N up rows and out = silu(gate) * up.
//
// The simple form: 32 x 32 tiles on CUDA cores.  Block y finds its group and rows by walking the offsets.
#include <cuda_runtime.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr int kTile = 32;

template <bool SWIGLU>
__global__ void __launch_bounds__(kTile * 8) grouped_kernel(const GroupedArgs a) {
    __shared__ float sx[kTile][kTile + 1], sw[SWIGLU ? 2 : 1][kTile][kTile + 1];
    pdl_launch_dependents();
    pdl_wait();
    int left = (int)blockIdx.y, lo = 0, hi = 0, e = 0;
    for (; e < a.groups; ++e) {
        lo = min(max(a.offsets[e], 0), a.P);
        hi = min(max(a.offsets[e + 1], lo), a.P);
        const int tiles = (hi - lo + kTile - 1) / kTile;
        if (left < tiles) break;
        left -= tiles;
    }
    if (e == a.groups) return;
    const int p0 = lo + left * kTile, n0 = (int)blockIdx.x * kTile;
    const int wide = SWIGLU ? 2 * a.N : a.N;
    const int c = threadIdx.x % kTile, r0 = threadIdx.x / kTile;
    const uint16_t *w = static_cast<const uint16_t *>(a.w) + (size_t)e * wide * a.K;
    const uint16_t *x = static_cast<const uint16_t *>(a.x);
    float acc[SWIGLU ? 2 : 1][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kTile) {
        __syncthreads();
        for (int r = r0; r < kTile; r += 8) {
            const bool in = k0 + c < a.K;
            const int p = min(p0 + r, hi - 1);
            const long long row = min(max(a.rows ? a.rows[p] : p, 0), a.x_rows - 1);
            sx[r][c] = in ? bf16_to_f32(x[row * a.K + k0 + c]) : 0.0f;
            for (int h = 0; h < (SWIGLU ? 2 : 1); ++h)
                sw[h][r][c] = in && n0 + r < a.N ? bf16_to_f32(w[(size_t)(h * a.N + n0 + r) * a.K + k0 + c]) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kTile; ++k)
            for (int i = 0; i < 4; ++i)
                for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) acc[h][i] = fmaf(sx[r0 + 8 * i][k], sw[h][c][k], acc[h][i]);
    }
    const uint16_t *bias = static_cast<const uint16_t *>(a.bias);
    if (n0 + c >= a.N) return;
    for (int i = 0; i < 4; ++i) {
        const int p = p0 + r0 + 8 * i;
        if (p >= hi) continue;
        float v = acc[0][i] + (bias ? bf16_to_f32(bias[(size_t)e * wide + n0 + c]) : 0.0f);
        if constexpr (SWIGLU) {
            const float up = acc[1][i] + (bias ? bf16_to_f32(bias[(size_t)e * wide + a.N + n0 + c]) : 0.0f);
            v = v / (1.0f + expf(-v)) * up;
        }
        static_cast<uint16_t *>(a.out)[(size_t)p * a.N + n0 + c] = f32_to_bf16(v);
    }
}

}  // namespace

int launch_grouped(const GroupedArgs &a, uint32_t flags, void *stream) {
    const long long tiles = (long long)a.P / kTile + (a.P < a.groups ? a.P : a.groups);
    if (tiles > 65535) return (int)cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + kTile - 1) / kTile), (unsigned)tiles);
    cfg.blockDim = dim3(kTile * 8);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, a.swiglu ? grouped_kernel<true> : grouped_kernel<false>, a);
}

}  // namespace bf16l
