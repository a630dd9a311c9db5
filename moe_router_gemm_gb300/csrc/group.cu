// group.cu — rows put in the order of their group (a routing's experts, requests' adapters), and a token's rows summed
// with their weights.
//
// Grouping is a stable counting sort of n small keys.  Each warp has a run of consecutive keys and a histogram of its own
// in shared memory; equal keys of a step of 32 find one another with match.any, so that a histogram has one writer and
// positions do not depend on timing.  The positions then follow from three sums: over the warps of a CTA, over the CTAs of
// the one cluster (through distributed shared memory), over the groups.
#include <cuda_runtime.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 32, kThreads = 32 * kWarps;
constexpr int kCluster = 8;

struct GroupArgs {
    const int32_t *ids;
    int32_t *offsets, *rows, *place;
    int n, k, groups;
    int cols;  // groups, and one more where what belongs to none is ordered behind them
    int per;   // keys of a warp, a multiple of 32
};

// Shared memory: the warps' histograms, the CTA's counts, the first position of each group's rows from this CTA.
__host__ __device__ constexpr int group_smem_bytes(int cols) { return 4 * cols * (kWarps + 2); }

__device__ __forceinline__ int key_of(const GroupArgs &a, int i, int end) {
    const int id = i < end ? __ldg(a.ids + i) : -1;
    return (unsigned)id < (unsigned)a.groups ? id : a.cols > a.groups && i < end ? a.groups : -1;
}

__global__ void __launch_bounds__(kThreads, 1) group_kernel(const GroupArgs a) {
    extern __shared__ int sm[];
    __shared__ int part[kWarps];
    int *count = sm + kWarps * a.cols, *start = count + a.cols;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)blockIdx.x, ctas = (int)gridDim.x;  // one cluster
    int *mine = sm + warp * a.cols;
    const long long lo64 = (long long)(rank * kWarps + warp) * a.per;
    const int lo = (int)(lo64 < a.n ? lo64 : a.n), hi = (int)(lo64 + a.per < a.n ? lo64 + a.per : a.n);

    for (int e = tid; e < kWarps * a.cols; e += kThreads) sm[e] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int key = key_of(a, i0 + lane, hi);
        const unsigned same = __match_any_sync(kAll, key);
        if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < a.cols; e += kThreads) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kWarps; ++w) {
            const int c = sm[w * a.cols + e];
            sm[w * a.cols + e] = sum;
            sum += c;
        }
        count[e] = sum;
    }
    cluster_sync();

    // groups up to 1024: one a thread
    auto counts = [&](int e, int &all, int &before) {
        for (int c = 0; c < ctas; ++c) {
            int v;
            asm volatile("ld.shared::cluster.u32 %0, [%1];"
                         : "=r"(v)
                         : "r"(mapa_shared(smem_u32(count + e), (uint32_t)c))
                         : "memory");
            all += v;
            before += c < rank ? v : 0;
        }
    };
    int all = 0, before = 0, none = 0, none_before = 0;
    if (tid < a.groups) counts(tid, all, before);
    if (tid == 0 && a.cols > a.groups) counts(a.groups, none, none_before);
    int upto = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) part[warp] = upto;
    cluster_sync();  // (and no CTA leaves while another reads its counts)
    int base = 0;
    for (int w = 0; w < warp; ++w) base += part[w];
    upto += base;
    if (tid < a.groups) {
        start[tid] = upto - all + before;
        if (rank == 0) {
            if (tid == 0) a.offsets[0] = 0;
            a.offsets[tid + 1] = upto;
        }
    }
    int kept = 0;
    for (int w = 0; w < kWarps; ++w) kept += part[w];
    if (tid == 0 && a.cols > a.groups) start[a.groups] = kept + none_before;
    __syncthreads();

    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane, key = key_of(a, i, hi);
        const unsigned same = __match_any_sync(kAll, key);
        int at = -1;
        if (key >= 0) at = start[key] + mine[key] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
        if (i < hi) {
            if (a.place) a.place[i] = at;
            if (at >= 0) a.rows[at] = i / a.k;
        }
    }
    if (a.cols > a.groups) return;
    for (long long p = kept + (long long)rank * kThreads + tid; p < a.n; p += (long long)ctas * kThreads) a.rows[p] = -1;
}

template <int BYTES>
struct Vec;
template <>
struct Vec<16> {
    using T = uint4;
};
template <>
struct Vec<8> {
    using T = uint2;
};
template <>
struct Vec<4> {
    using T = uint32_t;
};
template <>
struct Vec<2> {
    using T = uint16_t;
};

// out[t] = sum over j of weights[t][j] * y[place[t][j]] (+ addend[t]), one vector of BYTES a thread, in fp32, in the order
// of j, rounded once.
template <int BYTES>
__global__ void __launch_bounds__(256) combine_kernel(const uint16_t *__restrict__ y, const int32_t *__restrict__ place,
                                                      const float *__restrict__ weights,
                                                      const uint16_t *__restrict__ addend, uint16_t *__restrict__ out,
                                                      long long vectors, int per_row, int k, long long y_rows, int H) {
    using V = typename Vec<BYTES>::T;
    constexpr int n = BYTES / 2;
    pdl_launch_dependents();
    pdl_wait();
    for (long long v = (long long)blockIdx.x * blockDim.x + threadIdx.x; v < vectors; v += (long long)gridDim.x * blockDim.x) {
        const long long t = v / per_row, c = (v - t * per_row) * n;
        float sum[n];
#pragma unroll
        for (int i = 0; i < n; ++i) sum[i] = 0.0f;
        auto add = [&](const uint16_t *p, float w) {
            union {
                V v;
                uint16_t h[n];
            } u;
            u.v = *reinterpret_cast<const V *>(p);
#pragma unroll
            for (int i = 0; i < n; ++i) sum[i] = fmaf(w, bf16_to_f32(u.h[i]), sum[i]);
        };
        for (int j = 0; j < k; ++j) {
            const long long p = place[t * k + j];
            if (p >= 0 && p < y_rows) add(y + p * H + c, weights ? weights[t * k + j] : 1.0f);
        }
        if (addend) add(addend + t * H + c, 1.0f);
        union {
            V v;
            uint16_t h[n];
        } r;
#pragma unroll
        for (int i = 0; i < n; ++i) r.h[i] = f32_to_bf16(sum[i]);
        *reinterpret_cast<V *>(out + t * H + c) = r.v;
    }
}

template <int BYTES>
int launch_combine(const void *y, long long y_rows, const int32_t *place, const float *weights, const void *addend,
                   void *out, long long tokens, int k, int H, int num_sms, uint32_t flags, void *stream) {
    const int per_row = H / (BYTES / 2);
    const long long vectors = tokens * per_row, blocks = (vectors + 255) / 256, most = 8ll * num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(256);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, combine_kernel<BYTES>, static_cast<const uint16_t *>(y), place, weights,
                                   static_cast<const uint16_t *>(addend), static_cast<uint16_t *>(out), vectors, per_row, k,
                                   y_rows, H);
}

}  // namespace

int init_group() {
    return (int)cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     group_smem_bytes(kMaxGroups + 1));
}

int launch_group_rows(const int32_t *ids, int n, int k, int groups, bool rest, int32_t *offsets, int32_t *rows,
                      int32_t *place, uint32_t flags, void *stream) {
    const int ctas = n <= 4 * kThreads ? 1 : kCluster;
    const int warps = ctas * kWarps;
    GroupArgs a = {ids, offsets, rows, place, n, k, groups, groups + (rest ? 1 : 0), 0};
    a.per = (int)(((long long)n + warps - 1) / warps + 31) / 32 * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)group_smem_bytes(a.cols);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return (int)cudaLaunchKernelEx(&cfg, group_kernel, a);
}

int launch_combine_rows(const void *y, int64_t y_rows, const int32_t *place, const float *weights, const void *addend,
                        void *out, int64_t tokens, int k, int H, int num_sms, uint32_t flags, void *stream) {
    // rows of H elements: the widest vectors that every row of all three starts on
    const auto f = H % 8 == 0 ? launch_combine<16> : H % 4 == 0 ? launch_combine<8>
                   : H % 2 == 0 ? launch_combine<4> : launch_combine<2>;
    return f(y, y_rows, place, weights, addend, out, tokens, k, H, num_sms, flags, stream);
}

}  // namespace bf16l
