// group.cu — rows put in the order of their group (a routing's experts, requests' adapters), and a token's rows summed
// with their weights.
//
// Grouping is a stable counting sort of n small keys.  Each warp has a run of consecutive keys and a histogram of its own
// in shared memory; equal keys of a step of 32 find one another by ballots over the key's bits (match.any goes through the
// different keys one by one: 8192 x 8 keys of 256 groups 10.8 us, 7.7 so), so that a histogram has one writer and positions
// do not depend on timing.  It moves less than a megabyte: what bounds it is the chain of a launch, the ballots, three sums and
// two cluster barriers (16 x 8 keys in one CTA 2.6 us).  The positions then follow from three sums: over the warps of a CTA, over the CTAs of
// the one cluster (through distributed shared memory), over the groups.
#include <cuda_runtime.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 32, kThreads = 32 * kWarps;
constexpr int kCluster = 16;
constexpr int kKept = 4;  // steps whose keys a warp has in registers: all, up to 32 * kWarps * kCluster * kKept keys

struct GroupArgs {
    const int32_t *ids;
    int32_t *offsets, *rows, *place;
    int n, k, groups;
    int cols;  // groups, and one more where what belongs to none is ordered behind them
    int per;   // keys of a warp, a multiple of 32
    int bits;  // of a key, and of one more than the last
    int shift;  // log2 of k where k is a power of two, else -1
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
    pdl_wait();
    pdl_launch_dependents();  // (after the wait: the next kernel may rely on all that came before this one)

    // A step's key, and its place among the warp's of its group.
    auto count_step = [&](int key) {
        unsigned same = kAll;  // the lanes that have this key: bit by bit (no key: all bits of the width set, and past the last)
        for (int b = 0; b < a.bits; ++b) {
            const unsigned ones = __ballot_sync(kAll, (key >> b) & 1);
            same &= (key >> b) & 1 ? ones : ~ones;
        }
        const int at = key >= 0 ? mine[key] + __popc(same & ((1u << lane) - 1u)) : 0;
        __syncwarp();
        if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
        return at;
    };
    const bool kept_all = a.per <= 32 * kKept;
    int key[kKept], nth[kKept];
    for (int i0 = lo; i0 < hi; i0 += 32 * kKept) {  // (once where kept_all)
#pragma unroll
        for (int j = 0; j < kKept; ++j) key[j] = key_of(a, i0 + 32 * j + lane, hi);
#pragma unroll
        for (int j = 0; j < kKept; ++j)
            if (i0 + 32 * j < hi) nth[j] = count_step(key[j]);
    }
    __syncthreads();
    for (int e = tid; e < a.cols; e += kThreads) {
        int sum = 0;
        for (int w0 = 0; w0 < kWarps; w0 += 8) {
            int c[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) c[w] = sm[(w0 + w) * a.cols + e];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                sm[(w0 + w) * a.cols + e] = sum;
                sum += c[w];
            }
        }
        count[e] = sum;
    }
    cluster_sync();

    // groups up to 1024: one a thread
    int all = 0, before = 0, none_before = 0;
    if (ctas == 1) {
        if (tid < a.groups) all = count[tid];
    } else {
        auto counts = [&](int e, int &sum, int &earlier) {  // (all of a cluster's reads on their way together)
            int v[kCluster];
#pragma unroll
            for (int c = 0; c < kCluster; ++c)
                asm volatile("ld.shared::cluster.u32 %0, [%1];"
                             : "=r"(v[c])
                             : "r"(mapa_shared(smem_u32(count + e), (uint32_t)c)));
#pragma unroll
            for (int c = 0; c < kCluster; ++c) {
                sum += v[c];
                earlier += c < rank ? v[c] : 0;
            }
        };
        int none = 0;
        if (tid < a.groups) counts(tid, all, before);
        if (tid == 0 && a.cols > a.groups) counts(a.groups, none, none_before);
    }
    int upto = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) part[warp] = upto;
    cluster_sync();  // (and no CTA leaves while another reads its counts)
    int sums = part[lane];  // over the warps up to lane
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, sums, d);
        if (lane >= d) sums += v;
    }
    const int kept = __shfl_sync(kAll, sums, 31), base = __shfl_sync(kAll, sums, warp > 0 ? warp - 1 : 0);
    if (warp > 0) upto += base;
    if (tid < a.groups) {
        start[tid] = upto - all + before;
        if (rank == 0) {
            if (tid == 0) a.offsets[0] = 0;
            a.offsets[tid + 1] = upto;
        }
    }
    if (tid == 0 && a.cols > a.groups) start[a.groups] = kept + none_before;
    __syncthreads();

    // (`mine` is now the number of earlier warps' of each group)
    auto put = [&](int i, int key, int at) {
        if (i >= hi) return;
        if (a.place) a.place[i] = at;
        if (key >= 0) a.rows[at] = a.shift >= 0 ? i >> a.shift : i / a.k;
    };
    if (kept_all) {
#pragma unroll
        for (int j = 0; j < kKept; ++j)
            if (lo + 32 * j < hi) put(lo + 32 * j + lane, key[j], key[j] >= 0 ? start[key[j]] + mine[key[j]] + nth[j] : -1);
    } else {
        for (int i0 = lo; i0 < hi; i0 += 32) {
            const int k0 = key_of(a, i0 + lane, hi), at = count_step(k0);
            put(i0 + lane, k0, k0 >= 0 ? start[k0] + at : -1);
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

constexpr int kCombineThreads = 128, kAtOnce = 8;

// out[t] = sum over j of weights[t][j] * y[place[t][j]] (+ addend[t]), one vector of BYTES a thread, in fp32, in the order
// of j, rounded once.  HBM bounds it: every row of y is read once, by one thread for each of its vectors.  kAtOnce rows' loads
// go out before the first is used: 8192 x 8 x 7168 with an addend 180 us, 96% of the copy rate (275 one after the other).
// PER vectors a thread, kCombineThreads apart, where they are narrow (odd H): 6418 x 3 x 477 10 us (28 with one).
template <int BYTES, int PER>
__global__ void __launch_bounds__(kCombineThreads)
    combine_kernel(const uint16_t *__restrict__ y, const int32_t *__restrict__ place, const float *__restrict__ weights,
                   const uint16_t *__restrict__ addend, uint16_t *__restrict__ out, int blocks_per_row, int k,
                   long long y_rows, int H) {
    using V = typename Vec<BYTES>::T;
    constexpr int n = BYTES / 2;
    union U {
        V v;
        uint16_t h[n];
    };
    pdl_launch_dependents();
    pdl_wait();
    const long long t = blockIdx.x / blocks_per_row;
    const int c0 = ((int)(blockIdx.x - t * blocks_per_row) * kCombineThreads * PER + (int)threadIdx.x) * n;
    U last[PER];
    float sum[PER][n];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = c0 + q * kCombineThreads * n;
        if (addend && c < H) last[q].v = __ldg(reinterpret_cast<const V *>(addend + t * H + c));
#pragma unroll
        for (int i = 0; i < n; ++i) sum[q][i] = 0.0f;
    }
    for (int j0 = 0; j0 < k; j0 += kAtOnce) {
        U u[kAtOnce][PER];
        float w[kAtOnce];
        bool in[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const long long p = j0 + j < k ? __ldg(place + t * k + j0 + j) : -1;
            in[j] = p >= 0 && p < y_rows;
            if (in[j]) {
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    const int c = c0 + q * kCombineThreads * n;
                    if (c < H) u[j][q].v = __ldg(reinterpret_cast<const V *>(y + p * H + c));
                }
                w[j] = weights ? __ldg(weights + t * k + j0 + j) : 1.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (in[j]) {
#pragma unroll
                for (int q = 0; q < PER; ++q)
#pragma unroll
                    for (int i = 0; i < n; ++i) sum[q][i] = fmaf(w[j], bf16_to_f32(u[j][q].h[i]), sum[q][i]);
            }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = c0 + q * kCombineThreads * n;
        U r;
#pragma unroll
        for (int i = 0; i < n; ++i)
            r.h[i] = f32_to_bf16(addend ? sum[q][i] + bf16_to_f32(last[q].h[i]) : sum[q][i]);
        if (c < H) *reinterpret_cast<V *>(out + t * H + c) = r.v;
    }
}

template <int BYTES, int PER>
int launch_combine(const void *y, long long y_rows, const int32_t *place, const float *weights, const void *addend,
                   void *out, long long tokens, int k, int H, uint32_t flags, void *stream) {
    const int per_block = kCombineThreads * PER, blocks_per_row = (H / (BYTES / 2) + per_block - 1) / per_block;
    const long long most = 0x7FFFFFFFll / blocks_per_row;  // tokens of a launch
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    for (long long t = 0; t < tokens; t += most) {
        const long long now = tokens - t < most ? tokens - t : most;
        cfg.gridDim = dim3((unsigned)(now * blocks_per_row));
        const int r = (int)cudaLaunchKernelEx(
            &cfg, combine_kernel<BYTES, PER>, static_cast<const uint16_t *>(y), place + t * k, weights ? weights + t * k : nullptr,
            addend ? static_cast<const uint16_t *>(addend) + t * H : nullptr, static_cast<uint16_t *>(out) + t * H,
            blocks_per_row, k, y_rows, H);
        if (r) return r;
    }
    return 0;
}

}  // namespace

int init_group() {
    const int e = (int)cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            group_smem_bytes(kMaxGroups + 1));
    return e ? e : (int)cudaFuncSetAttribute(group_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

int launch_group_rows(const int32_t *ids, int n, int k, int groups, bool rest, int32_t *offsets, int32_t *rows,
                      int32_t *place, uint32_t flags, void *stream) {
    // One CTA up to two steps of all its warps, else all of a cluster (256 groups: 1100 keys 4.9 us in one, 5.4 in 16; 2048 5.5
    // both; 4096 7.9 and 5.5).  The kernel takes no other numbers.
    const int ctas = n <= 2 * kThreads ? 1 : kCluster;
    const int warps = ctas * kWarps;
    GroupArgs a = {ids, offsets, rows, place, n, k, groups, groups + (rest ? 1 : 0), 0, 1, -1};
    for (int s = 0; s < 31; ++s)
        if (k == 1 << s) a.shift = s;
    while ((1 << a.bits) <= a.cols) ++a.bits;  // (-1 then differs from every key)
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
                        void *out, int64_t tokens, int k, int H, uint32_t flags, void *stream) {
    // rows of H elements: the widest vectors that every row of all three starts on
    const auto f = H % 8 == 0 ? launch_combine<16, 1> : H % 4 == 0 ? launch_combine<8, 2>
                   : H % 2 == 0 ? launch_combine<4, 4> : launch_combine<2, 4>;
    return f(y, y_rows, place, weights, addend, out, tokens, k, H, flags, stream);
}

}  // namespace bf16l
