// mxfp4.cu — MXFP4: the quantisation of bf16 rows, the values of codes, and the
// block-scaled linear on warp-level tensor-core MMAs.
//
// Quantisation: four lanes hold a 32-element block, eight values each; the
// block's largest magnitude by a quad shuffle on the bf16 bits, the scale
// exponent from its exponent field, one exact multiplication by 2^-s and the
// hardware's e2m1 conversion (nearest even, saturating) per value.  2 bytes in
// and 0.53 out per element: bound by HBM.
//
// Linear: one mma.sync.m16n8k32 e4m3 step is one scale block.
//   * grid (S, ceil(N/8), ceil(M/16)), clusters of S CTAs along K; CTA (r, q, z)
//     owns W rows 8q..8q+7, tokens 16z..16z+15 and the r-th of S runs of blocks,
//     which its warps split;
//   * lane (g, t) loads 4 bytes of W row g and of x rows g and g+8: codes 32b +
//     8t .. +8 of block b, widened to e4m3 in registers (every value times 2^-6,
//     exact); even codes feed the MMA's k 4t..4t+3, odd ones k 16+4t.., the same
//     permutation for both operands;
//   * a block's sum has at most 13 significant bits and is exact; it is scaled
//     by its two block scales (powers of two; carrying the codes' 2^-12 keeps
//     the intermediate inside fp32 for every pair of scale bytes) and added to
//     the running fp32 sum, which is multiplied by 2^12 at the end;
//   * warps' sums in warp order in shared memory; ranks 1..S-1 send theirs to
//     rank 0 with st.async counted on its mbarrier; rank 0 sums in rank order,
//     adds bias, rounds, stores: the order never changes.
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

constexpr int kM4Warps = 8;
constexpr int kM4U = 4;  // blocks per lane per batch
constexpr int kM4MaxCluster = 16;

__global__ void __launch_bounds__(256) quant_mxfp4_kernel(const uint4 *__restrict__ x, uint32_t *__restrict__ q,
                                                          uint8_t *__restrict__ scales, long long nvec) {
    pdl_launch_dependents();
    pdl_wait();  // x may be written by the previous kernel
    const long long stride = (long long)gridDim.x * blockDim.x;
    const unsigned quad = 0xFu << (threadIdx.x & 28u);
    // nvec and the stride are multiples of 4: a quad is in or out of the loop together
    for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
        uint32_t sb;
        q[v] = mxfp4_quant_vec(__ldg(x + v), quad, sb);
        if ((threadIdx.x & 3) == 0) scales[v >> 2] = (uint8_t)sb;
    }
}

__global__ void __launch_bounds__(256) dequant_mxfp4_kernel(const uint32_t *__restrict__ q,
                                                            const uint8_t *__restrict__ scales, uint4 *__restrict__ out,
                                                            long long nvec) {
    pdl_launch_dependents();
    pdl_wait();
    const long long stride = (long long)gridDim.x * blockDim.x;
    for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < nvec; v += stride) {
        const uint32_t w = __ldg(q + v);
        const float s = e8m0_value(__ldg(scales + (v >> 2)));
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // the code's fields at bf16's places read as the value times 2^-126
            const uint32_t c = w >> (4 * j);
            f[j] = (__uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f) * s;
        }
        out[v] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                            pack_bf16x2(f[6], f[7]));
    }
}

template <bool HI>
__global__ void __launch_bounds__(kM4Warps * 32)
    mxfp4_linear_kernel(const uint8_t *__restrict__ xq, const uint8_t *__restrict__ xs,
                        const uint8_t *__restrict__ wq, const uint8_t *__restrict__ ws,
                        const uint16_t *__restrict__ bias, uint16_t *__restrict__ out, int M, int N, int K, int S,
                        int32_t *status, int w_early) {
    __shared__ float4 part[kM4Warps][32];
    __shared__ float4 recv[kM4MaxCluster][32];
    __shared__ __align__(8) uint64_t rbar;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int nw = (int)blockDim.x >> 5;
    const int nb = K >> 5;
    const size_t pitch = (size_t)(K >> 1);  // bytes of codes per row
    {
        const int m0 = 16 * (int)blockIdx.z;
        xq += (size_t)m0 * pitch;
        xs += (size_t)m0 * nb;
        out += (size_t)m0 * N;
        M = (M - m0) < 16 ? (M - m0) : 16;
    }
    const bool clus = S > 1;
    const int rank = clus ? (int)cluster_ctarank() : 0;
    const int n0 = 8 * (int)blockIdx.y;
    const int cb0 = mul_div(nb, rank, S), cb1 = mul_div(nb, rank + 1, S);
    const int b0 = cb0 + mul_div(cb1 - cb0, warp, nw), b1 = cb0 + mul_div(cb1 - cb0, warp + 1, nw);
    if (!w_early) pdl_wait();
    const bool tok_lo = g < M, tok_hi = HI && (g + 8 < M);
    const int row = n0 + g;
    const int na = n0 + 2 * t, nc = na + 1;
    const uint8_t *wr = wq + (size_t)(row < N ? row : N - 1) * pitch + 4 * t;
    const uint8_t *xlo = xq + (size_t)(tok_lo ? g : 0) * pitch + 4 * t;
    const uint8_t *xhi = xq + (size_t)(tok_hi ? g + 8 : 0) * pitch + 4 * t;
    const uint8_t *wsa = ws + (size_t)(na < N ? na : N - 1) * nb, *wsb = ws + (size_t)(nc < N ? nc : N - 1) * nb;
    const uint8_t *xsl = xs + (size_t)(tok_lo ? g : 0) * nb, *xsh = xs + (size_t)(tok_hi ? g + 8 : 0) * nb;

    uint32_t wv[kM4U], swa[kM4U], swb[kM4U];
    auto load_w = [&](int bb) {
#pragma unroll
        for (int u = 0; u < kM4U; ++u) {
            const int b = bb + u;
            const bool in = b < b1;
            wv[u] = in ? __ldg(reinterpret_cast<const uint32_t *>(wr + 16 * (size_t)b)) : 0u;
            swa[u] = in ? __ldg(wsa + b) : 127u;
            swb[u] = in ? __ldg(wsb + b) : 127u;
        }
    };
    load_w(b0);

    if (tid == 0) {
        mbar_init(&rbar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (clus) cluster_arrive_relaxed();  // phase 1: "my receive barrier is initialised"
    pdl_launch_dependents();
    pdl_wait();

    float c[4] = {0.f, 0.f, 0.f, 0.f};
    for (int bb = b0; bb < b1; bb += kM4U) {
        if (bb != b0) load_w(bb);
        uint32_t al[kM4U], ah[kM4U], sxl[kM4U], sxh[kM4U];
#pragma unroll
        for (int u = 0; u < kM4U; ++u) {
            const int b = bb + u;
            const bool in = b < b1;
            al[u] = (tok_lo && in) ? __ldg(reinterpret_cast<const uint32_t *>(xlo + 16 * (size_t)b)) : 0u;
            ah[u] = (HI && tok_hi && in) ? __ldg(reinterpret_cast<const uint32_t *>(xhi + 16 * (size_t)b)) : 0u;
            sxl[u] = in ? __ldg(xsl + b) : 127u;
            sxh[u] = (HI && in) ? __ldg(xsh + b) : 127u;
        }
#pragma unroll
        for (int u = 0; u < kM4U; ++u) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t a0, a1 = 0, a2, a3 = 0, w0, w1;
            e2m1_to_e4m3(al[u], a0, a2);
            if (HI) e2m1_to_e4m3(ah[u], a1, a3);
            e2m1_to_e4m3(wv[u], w0, w1);
            mma_m16n8k32_e4m3(d, a0, a1, a2, a3, w0, w1);
            const float fl = e8m0_value(sxl[u]), fh = e8m0_value(sxh[u]);
            const float fa = e8m0_value(swa[u]), fb = e8m0_value(swb[u]);
            c[0] += (d[0] * fl) * fa;
            c[1] += (d[1] * fl) * fb;
            c[2] += (d[2] * fh) * fa;
            c[3] += (d[3] * fh) * fb;
        }
    }
    part[warp][lane] = make_float4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (warp == 0) {
        for (int w = 0; w < nw; ++w) {  // warps in order
            const float4 p = part[w][lane];
            s.x += p.x;
            s.y += p.y;
            s.z += p.z;
            s.w += p.w;
        }
    }
    bool have = true;
    if (clus) {
        cluster_wait_acquire();  // phase 1 done: rank 0's receive barrier exists
        if (rank != 0) {
            if (warp == 0)
                st_async_f4(mapa_shared(smem_u32(&recv[rank][lane]), 0), s.x, s.y, s.z, s.w,
                            mapa_shared(smem_u32(&rbar), 0));
        } else {
            if (tid == 0) mbar_arrive_expect_tx(&rbar, (uint32_t)((S - 1) * 32 * 16));
            if (warp == 0) {
                have = mbar_wait_cluster(&rbar, 0, status, kSiteRecv);
                for (int r = 1; r < S; ++r) {  // ranks in order
                    const float4 p = recv[r][lane];
                    s.x += p.x;
                    s.y += p.y;
                    s.z += p.z;
                    s.w += p.w;
                }
            }
        }
        cluster_arrive_relaxed();  // phase 2: everything rank 0 receives has landed
    }
    if (rank == 0 && warp == 0 && have) {
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = g + (j >> 1) * 8, n = n0 + 2 * t + (j & 1);
            if (m < M && n < N) {
                float r = v[j] * 4096.0f;
                if (bias) r += bf16_to_f32(bias[n]);
                out[(size_t)m * N + n] = f32_to_bf16(r);
            }
        }
    }
    if (clus) cluster_wait_acquire();  // phase 2 done: rank 0 holds every partial; all may exit
}

using M4Fn = void (*)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, const uint16_t *, uint16_t *,
                      int, int, int, int, int32_t *, int);

M4Fn pick_m4(int M) { return M > 8 ? mxfp4_linear_kernel<true> : mxfp4_linear_kernel<false>; }

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

int init_mxfp4() {
    for (int M : {8, 16}) {
        const int e = (int)cudaFuncSetAttribute(pick_m4(M), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e) return e;
    }
    return 0;
}

int launch_mxfp4(const void *xq, const void *xs, const void *wq, const void *ws, const void *bias, void *out, int M,
                 int N, int K, int S, int threads, uint32_t flags, void *stream, int32_t *status) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S, (unsigned)((N + 7) / 8), (unsigned)((M + 15) / 16));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, pick_m4(M), static_cast<const uint8_t *>(xq), static_cast<const uint8_t *>(xs),
                                   static_cast<const uint8_t *>(wq), static_cast<const uint8_t *>(ws),
                                   static_cast<const uint16_t *>(bias), static_cast<uint16_t *>(out), M, N, K, S,
                                   status, w_early_of(flags));
}

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
