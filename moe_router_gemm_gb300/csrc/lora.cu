// lora.cu — the low-rank adapters' share of a linear for few rows: h = x @ A_a^T for each row's adapter a, then
// out = y + scale_a * h @ B_a^T, with y the shared projection in fp32, by the dense linear's own kernels between the two.
//
// Both kernels stand for little work (131 KB of an adapter of rank 16 and 4096 columns each way) and much latency, so each
// spreads over the SMs: the inner one takes four ranks of a row a block, and splits K over more blocks as long as all are
// resident at once; the outer one adds those sums, and the projection's where that comes in parts, in order, when it reads
// them.  Up to 64 rows the inner one also asks L2 for B_a (more rows ask for the same ones: 128 x 14336 x 4096 r16 46.2 us,
// 43.8 without), and the outer one has its rows of B on their way before it waits for the projection.  61 x 2112 x 7168 with
// rank 32: 18.3 us, of which the projection alone takes 10.9; 8 x 4096 x 4096 with rank 16 10.4 (6.6), 64 x 4096 x 4096 with
// rank 64 26.0.
#include <cuda_runtime.h>

#include "grouped.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr int kRanks = 4;  // of a block of the inner kernel
constexpr int kOuterThreads = 128, kOuterBlocks = 9;
// (A warp has at least four loads of 512 bytes in flight.)
__host__ __device__ constexpr int outer_sets(int g) { return g < 4 ? 4 / g : 1; }

// A block sums kRanks ranks of a row over a part of K, its warps taking 256 elements in turn.  Eight warps of a block and
// parts of K in multiples of 256 took 0.5 to 1 us less than four warps and multiples of 1024 (8 x 4096 x 4096 r16 11.3 -> 10.3
// us, 61 x 2112 x 7168 r32 20.0 -> 19.1) where the blocks are few, and 1 to 5 us more where they are many (inner_warps); eight
// ranks a block, sixteen warps or more registers were slower.
template <int kInnerWarps>
__global__ void __launch_bounds__(32 * kInnerWarps) lora_inner_kernel(const LoraArgs a) {
    __shared__ float part[kInnerWarps][kRanks];
    // The next kernel may start once this one has waited: it then reads nothing but h that could still be written.  Where the
    // rows are ordered by adapter, the kernel before is the one that orders them, which has waited for all others and which
    // nothing here depends on: the two run side by side, and one block waits for it at the end, for whoever waits for this
    // one (256 x 14336 x 4096 r16 50.2 -> 47.2 us; asking L2 for B's rows there, 26 MB, took 2 us more).
    if (a.splits) pdl_wait();
    pdl_launch_dependents();
    const bool last = !a.splits && (blockIdx.x | blockIdx.z) == 0;
    const int t = blockIdx.x, s = blockIdx.y, splits = (int)gridDim.y, r0 = kRanks * (int)blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = __ldg(a.ids + t);
    if (a.span && threadIdx.x == 0 && (blockIdx.x | blockIdx.y | blockIdx.z) == 0) {
        a.span[0] = 0;
        a.span[1] = a.M;
    }
    if ((unsigned)id >= (unsigned)a.L) {  // (its inner values are not read)
        if (last) pdl_wait();
        return;
    }
    if (threadIdx.x == 0 && a.splits && !a.span) {  // this block's part of B's rows, for the outer kernel
        const int blocks = splits * (int)gridDim.z, i = s + splits * (int)blockIdx.z;
        const int n0 = (int)((long long)a.N * i / blocks), n1 = (int)((long long)a.N * (i + 1) / blocks);
        const uint16_t *b = static_cast<const uint16_t *>(a.b) + ((size_t)id * a.N + n0) * a.R;
        const long long bytes = (long long)(n1 - n0) * a.R * 2;
        prefetch_l2(b, (uint32_t)(bytes < (1 << 20) ? bytes : 1 << 20));
    }
    constexpr int kStep = 256 * kInnerWarps;
    const int each = ((a.K + splits - 1) / splits + 255) / 256 * 256, k0 = min(s * each, a.K), k1 = min(k0 + each, a.K);
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
        if (a.splits) {  // (a part of the sum: the scale, which could overflow it, comes with the whole)
            static_cast<float *>(a.h)[((size_t)s * a.M + t) * a.R + r0 + r] = v;
        } else {
            if (a.scale) v *= __ldg(a.scale + id);
            uint32_t high, low;
            two_bf16(v, high, low);
            uint16_t *h = static_cast<uint16_t *>(a.h) + (size_t)t * 2 * a.R + r0 + r;
            h[0] = (uint16_t)high;
            h[a.R] = (uint16_t)low;
        }
    }
    if (last) pdl_wait();
}

// A row of B (R values) goes to G lanes, G being the power of two from R / 8 up, 16 bytes each, so that a warp reads 512
// contiguous bytes at a time (where R / 8 is G); G such steps give each lane G parts of G outputs, and exchanging halves of
// them log2(G) times leaves each lane the sum of one.  The rows of B are on their way while the shared product still runs
// (which started when the inner kernel had waited for all before it).  With an output a thread and its row of B in one lane
// 61 x 2112 x 7168 r32 took 18.6 us (18.2 so), 64 x 4096 x 4096 r64 30.9 (27.5), 64 x 7168 x 7168 r128 71 (56).
template <int G>
__global__ void __launch_bounds__(kOuterThreads) lora_outer_kernel(const LoraArgs a) {
    constexpr int kSets = outer_sets(G), kRows = 32 / G;  // sets of 32 outputs; rows of B in a step
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, p = lane & (G - 1), q = lane / G;
    const int t = blockIdx.x, id = __ldg(a.ids + t);
    const bool has = (unsigned)id < (unsigned)a.L && 8 * p < a.R;  // (R % 8 == 0)
    const uint16_t *B = static_cast<const uint16_t *>(a.b) + (has ? (size_t)id * a.N * a.R + 8 * p : 0);
    const unsigned N = (unsigned)a.N, step = gridDim.y * (kSets * kOuterThreads);  // (together below 2^32)
    unsigned n = (blockIdx.y * (kOuterThreads / 32) + (threadIdx.x >> 5)) * (32 * kSets) + q;
    uint4 v[kSets][G];
    auto load = [&]() {
        const uint16_t *row = B + (size_t)n * a.R;
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int i = 32 * s + j * kRows;
                v[s][j] = has && n + i < N ? __ldg(reinterpret_cast<const uint4 *>(row + i * a.R)) : make_uint4(0, 0, 0, 0);
            }
    };
    load();
    const float f = has && a.scale ? __ldg(a.scale + id) : 1.0f;
    pdl_wait();
    float h[8] = {};
    if (has) {
        const float4 *hs = reinterpret_cast<const float4 *>(static_cast<const float *>(a.h) + (size_t)t * a.R + 8 * p);
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s, hs += (size_t)a.M * a.R / 4) {
            const float4 lo = hs[0], hi = hs[1];
            h[0] += lo.x, h[1] += lo.y, h[2] += lo.z, h[3] += lo.w;
            h[4] += hi.x, h[5] += hi.y, h[6] += hi.z, h[7] += hi.w;
        }
    }
    if (a.scale) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= f;
    }
    const float *from = a.y + (size_t)t * a.pitch;
    const size_t plane = (size_t)a.M * a.pitch;
    uint16_t *to = static_cast<uint16_t *>(a.out) + (size_t)t * N;
    for (; n - q < N; n += step, load()) {
        float y[kSets];
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const unsigned i = n + 32 * s + p * kRows;
            y[s] = 0.0f;
#pragma unroll 4
            for (int k = 0; i < N && k < a.parts; ++k) y[s] += from[k * plane + i];
        }
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            float d[G];
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const uint4 b = v[s][j];
                d[j] = h[0] * bf16_lo(b.x);
                d[j] = fmaf(h[1], bf16_hi(b.x), d[j]);
                d[j] = fmaf(h[2], bf16_lo(b.y), d[j]);
                d[j] = fmaf(h[3], bf16_hi(b.y), d[j]);
                d[j] = fmaf(h[4], bf16_lo(b.z), d[j]);
                d[j] = fmaf(h[5], bf16_hi(b.z), d[j]);
                d[j] = fmaf(h[6], bf16_lo(b.w), d[j]);
                d[j] = fmaf(h[7], bf16_hi(b.w), d[j]);
            }
#pragma unroll
            for (int w = G / 2; w; w >>= 1)
#pragma unroll
                for (int j = 0; j < w; ++j) {
                    const bool upper = lane & w;
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? d[j] : d[j + w], w);
                    d[j] = (upper ? d[j + w] : d[j]) + other;
                }
            const unsigned i = n + 32 * s + p * kRows;
            if (i < N) to[i] = f32_to_bf16(y[s] + d[0]);
        }
    }
}

// One or two rows: a warp for each W row, its first kAhead vectors of W, and B's row, on their way while the inner kernel
// still runs (which has let this one start when all kernels before it were done); then the row's h, and one sum over the
// warp for the shared product and the adapter's.  x in shared memory.  1 x 4096 x 4096 with rank 16 8.3 us (floor 5.0; 9.9
// with the dense linear's kernel and the outer one), 1 x 2112 x 7168 with rank 32 8.6 (11.3), 1 x 1024 x 1024 3.2 (5.7).
// Three or four rows took longer so than by the other form, 16 vectors ahead (which halve the resident warps) 11.1, and one
// kernel whose clusters of eight CTAs each work the inner values out 9.0.
constexpr int kRowWarps = 8, kAhead = 8;
template <int M>
__global__ void __launch_bounds__(32 * kRowWarps, 4) lora_rows_kernel(const LoraArgs a, const uint16_t *__restrict__ w,
                                                                   const uint16_t *__restrict__ bias) {
    extern __shared__ uint4 sx[];
    const int lane = threadIdx.x & 31, n = (int)blockIdx.x * kRowWarps + (int)(threadIdx.x >> 5);
    const int vectors = a.K / 8;  // (K % 8 == 0)
    const bool in = n < a.N;
    const uint4 *row = reinterpret_cast<const uint4 *>(w + (size_t)(in ? n : 0) * a.K);
    uint4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (in && 32 * i + lane < vectors) v[i] = ldg_stream_v4(row + 32 * i + lane);
    const uint4 *x = static_cast<const uint4 *>(a.x);
    for (int i = threadIdx.x; i < M * vectors; i += 32 * kRowWarps) sx[i] = __ldg(x + i);
    int id[M];
    float f[M], b[M][kLoraMaxRank / 32];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        id[m] = __ldg(a.ids + m);
        const bool has = in && (unsigned)id[m] < (unsigned)a.L;
        f[m] = has && a.scale ? __ldg(a.scale + id[m]) : 1.0f;
#pragma unroll
        for (int q = 0; q < kLoraMaxRank / 32; ++q) {
            const int r = 32 * q + lane;
            b[m][q] = has && r < a.R ? bf16_to_f32(__ldg(static_cast<const uint16_t *>(a.b) +
                                                         ((size_t)id[m] * a.N + n) * a.R + r))
                                     : 0.0f;
        }
    }
    const float extra = in && bias ? bf16_to_f32(__ldg(bias + n)) : 0.0f;
    __syncthreads();
    pdl_launch_dependents();
    float sum[M] = {};
    auto add = [&](const uint4 &q, int k) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const uint4 xv = sx[m * vectors + k];
            sum[m] = fma2_bf16(xv.x, q.x, sum[m]);
            sum[m] = fma2_bf16(xv.y, q.y, sum[m]);
            sum[m] = fma2_bf16(xv.z, q.z, sum[m]);
            sum[m] = fma2_bf16(xv.w, q.w, sum[m]);
        }
    };
    if (in) {
        for (int k0 = 0; k0 < vectors; k0 += 32 * kAhead) {
            const int next = k0 + 32 * kAhead;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = k0 + 32 * i + lane;
                if (k < vectors) add(v[i], k);
                if (next + 32 * i + lane < vectors) v[i] = ldg_stream_v4(row + next + 32 * i + lane);
            }
        }
    }
    pdl_wait();  // the inner values
#pragma unroll
    for (int m = 0; m < M; ++m) {
        if ((unsigned)id[m] >= (unsigned)a.L) continue;
#pragma unroll
        for (int q = 0; q < kLoraMaxRank / 32; ++q) {
            const int r = 32 * q + lane;
            if (r >= a.R) continue;
            float h = 0.0f;
#pragma unroll 4
            for (int s = 0; s < a.splits; ++s) h += static_cast<const float *>(a.h)[((size_t)s * M + m) * a.R + r];
            sum[m] = fmaf(f[m] * h, b[m][q], sum[m]);
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
        for (int d = 16; d; d >>= 1) sum[m] += __shfl_xor_sync(0xFFFFFFFFu, sum[m], d);
        if (in && lane == m) static_cast<uint16_t *>(a.out)[(size_t)m * a.N + n] = f32_to_bf16(sum[m] + extra);
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

// Warps of a block of the inner kernel: eight up to two waves of blocks (65 x 4096 x 4096 r16 30.9 us, 32.0 with four), four
// above (1024 x 2048 x 2048 r16 28.3, 33.0 with eight; 435 x 377 x 5944 r32 38.9 and 41.8).
int inner_warps(int M, int R) { return (long long)M * (R / kRanks) <= 8 * kGb300Sms ? 8 : 4; }

}  // namespace

// Parts of K: as many as leave all blocks resident at once (four an SM), each long enough for the warps of a block.
int lora_splits(int M, int K, int R) {
    const int blocks = M * (R / kRanks), want = 4 * kGb300Sms / blocks;  // (few rows)
    const int each = 256 * inner_warps(M, R), most = (K + each - 1) / each, s = want < most ? want : most;
    return s < 1 ? 1 : s > 8 ? 8 : s;
}

int launch_lora_inner(const LoraArgs &a, uint32_t flags, void *stream) {
    const dim3 grid((unsigned)a.M, (unsigned)(a.splits ? a.splits : 1), (unsigned)(a.R / kRanks));
    const int warps = inner_warps(a.M, a.R);
    return launch(warps == 8 ? lora_inner_kernel<8> : lora_inner_kernel<4>, grid, 32 * warps, a, flags, stream);
}

int init_lora() {
    for (auto f : {lora_rows_kernel<1>, lora_rows_kernel<2>}) {
        const int e = (int)cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kLoraRowsSmem);
        if (e) return e;
    }
    return 0;
}

int launch_lora_rows(const LoraArgs &a, const void *w, const void *bias, uint32_t flags, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + kRowWarps - 1) / kRowWarps));
    cfg.blockDim = dim3(32 * kRowWarps);
    cfg.dynamicSmemBytes = (size_t)a.M * a.K * 2;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, a.M == 1 ? lora_rows_kernel<1> : lora_rows_kernel<2>, a,
                                   static_cast<const uint16_t *>(w), static_cast<const uint16_t *>(bias));
}

int launch_lora_outer(const LoraArgs &a, uint32_t flags, void *stream) {
    int g = 1;
    while (8 * g < a.R) g *= 2;
    const int outputs = outer_sets(g) * kOuterThreads, blocks = (int)(((long long)a.N + outputs - 1) / outputs);
    // Blocks for one wave, each going on along N: 64 x 7168 x 7168 r128 51.7 us, 53.9 with a block for every 128 outputs, 64 x
    // 14336 x 4096 r16 36.3 and 37.0.
    const int wave = kOuterBlocks * kGb300Sms / a.M, most = wave > 1 ? wave : 1;
    const dim3 grid((unsigned)a.M, (unsigned)(blocks < most ? blocks : most));
    auto f = g == 1 ? lora_outer_kernel<1> : g == 2 ? lora_outer_kernel<2> : g == 4 ? lora_outer_kernel<4>
           : g == 8 ? lora_outer_kernel<8> : lora_outer_kernel<16>;
    return launch(f, grid, kOuterThreads, a, flags, stream);
}

}  // namespace bf16l
