// mxfp4.cu — MXFP4: the quantisation of bf16 rows, and the values of codes.
//
// Four lanes hold a 32-element block, eight values each; the block's largest
// magnitude by a quad shuffle on the bf16 bits, the scale exponent from its exponent
// field, one exact multiplication by 2^-s and the hardware's e2m1 conversion (nearest
// even, saturating) per value.  2 bytes in and 0.53 out per element, and the reverse:
// bound by HBM.  7168 x 7168: 19.4 us quantised (98% of the copy bandwidth; 22.7 with
// loads that also fill L1), 22.3 us back (86%).
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

__global__ void __launch_bounds__(256) quant_mxfp4_kernel(const uint4 *__restrict__ x, uint32_t *__restrict__ q,
                                                          uint8_t *__restrict__ scales, long long nvec) {
    pdl_launch_dependents();
    pdl_wait();  // x may be written by the previous kernel
    const long long stride = (long long)gridDim.x * blockDim.x;
    const unsigned quad = 0xFu << (threadIdx.x & 28u);
    // nvec and the stride are multiples of 4: a quad is in or out of the loop together
    for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
        uint32_t sb;
        q[v] = mxfp4_quant_vec(ldg_stream_v4(x + v), quad, sb);
        if ((threadIdx.x & 3) == 0) scales[v >> 2] = (uint8_t)sb;
    }
}

constexpr int kUnroll = 2;  // vectors of a thread whose loads go out together

__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint32_t *__restrict__ q,
                                                            const uint8_t *__restrict__ scales, uint4 *__restrict__ out,
                                                            long long nvec) {
    pdl_launch_dependents();
    pdl_wait();
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long v0 = (long long)blockIdx.x * blockDim.x + threadIdx.x; v0 < nvec; v0 += kUnroll * stride) {
        uint32_t w[kUnroll], e[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const long long v = v0 + k * stride;
            if (v < nvec) w[k] = __ldg(q + v), e[k] = __ldg(scales + (v >> 2));
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const long long v = v0 + k * stride;
            if (v >= nvec) break;
            const float s = e8m0_value(e[k]);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // the code's fields at fp32's places read as the value times 2^-126
                const uint32_t c = w[k] >> (4 * j);
                f[j] = (__uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f) * s;
            }
            out[v] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                pack_bf16x2(f[6], f[7]));
        }
    }
}

cudaLaunchConfig_t stream_config(long long items, int threads, int per_sm, int num_sms, uint32_t flags, void *stream,
                                 cudaLaunchAttribute *attr) {
    long long blocks = (items + threads - 1) / threads;
    const long long cap = (long long)per_sm * num_sms;
    if (blocks > cap) blocks = cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = (cudaStream_t)stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

int launch_quant_mxfp4(const void *x, void *q, void *scales, long long n, int num_sms, uint32_t flags, void *stream) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = stream_config(n / 8, 256, 8, num_sms, flags, stream, attr);
    return (int)cudaLaunchKernelEx(&cfg, quant_mxfp4_kernel, static_cast<const uint4 *>(x),
                                   static_cast<uint32_t *>(q), static_cast<uint8_t *>(scales), n / 8);
}

int launch_dequant_mxfp4(const void *q, const void *scales, void *out, long long n, int num_sms, uint32_t flags,
                         void *stream) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = stream_config(n / 8, 256, 8, num_sms, flags, stream, attr);
    return (int)cudaLaunchKernelEx(&cfg, dequant_mxfp4_kernel, static_cast<const uint32_t *>(q),
                                   static_cast<const uint8_t *>(scales), static_cast<uint4 *>(out), n / 8);
}

}  // namespace bf16l
