// route.cu — the k experts of each token and their weights from the router's
// logits: softmax or sigmoid scores, a bias for the choice alone, limited groups,
// top-k, renormalised weights.
//
// One warp per token.  A key is an unsigned word whose order is the float's
// (NaN and -inf at the bottom, -0 equal to +0, 0 for an expert that a group
// limit or an earlier pick took out), so a pick is two warp reductions: the
// largest key, then the lowest expert that has it.
#include <cuda_runtime.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

struct RouteArgs {
    const void *logits;
    const float *bias;
    float *weights;
    int32_t *ids;
    long long tokens, ld;
    int E, k, groups, top_groups, group_best, softmax, renorm, bf16;
    float scale;
};

constexpr unsigned kAll = 0xFFFFFFFFu;

// Order-preserving key: a < b as floats <=> key(a) < key(b); -0 as +0; NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
    v = (v != v) ? -INFINITY : v + 0.0f;
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
// ... and back.
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ (~(uint32_t)((int32_t)k >> 31) | 0x80000000u));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

__device__ __forceinline__ float load_logit(const RouteArgs &a, long long at) {
    return a.bf16 ? bf16_to_f32(static_cast<const uint16_t *>(a.logits)[at]) : static_cast<const float *>(a.logits)[at];
}

// VPL: experts per lane; expert e sits in slot e / 32 of lane e % 32.
template <int VPL>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tok < a.tokens; tok += warps) {
        const long long at = tok * a.ld;
        float l[VPL];
        uint32_t key[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = 32 * j + lane;
            l[j] = e < a.E ? load_logit(a, at + e) : -INFINITY;
        }
        float mx = 0.0f, total = 0.0f;
        if (a.softmax) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < VPL; ++j) m = fmaxf(m, l[j]);
            mx = key_value(__reduce_max_sync(kAll, order_key(m)));
            if (mx == -INFINITY) mx = 0.0f;  // every expert is out: exp(-inf) = 0 throughout
#pragma unroll
            for (int j = 0; j < VPL; ++j) total += expf(l[j] - mx);
            total = warp_sum(total);
        }
        const bool by_logit = a.softmax && !a.bias && a.group_best == 1;
        auto score = [&](float v) {
            if (a.softmax) return total == 0.0f ? 0.0f : expf(v - mx) / total;
            return 1.0f / (1.0f + expf(-v));
        };
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = 32 * j + lane;
            float v = l[j];
            if (e < a.E && !by_logit && v != -INFINITY) v = score(v) + (a.bias ? __ldg(a.bias + e) : 0.0f);
            key[j] = e < a.E ? order_key(v) : 0u;
        }
        if (a.groups > 1) {
            const int each = a.E / a.groups;
            uint32_t gkey = 0;  // lane g: the key of group g
            for (int g = 0; g < a.groups; ++g) {
                const int e0 = g * each, e1 = e0 + each;
                float sum = 0.0f;
                uint32_t taken = ~0u;  // the expert that gave the largest key
                for (int b = 0; b < a.group_best; ++b) {
                    uint32_t best = 0;
                    int who = INT_MAX;
#pragma unroll
                    for (int j = 0; j < VPL; ++j) {
                        const int e = 32 * j + lane;
                        if (e >= e0 && e < e1 && (uint32_t)e != taken && key[j] > best) best = key[j], who = e;
                    }
                    const uint32_t top = __reduce_max_sync(kAll, best);
                    taken = (uint32_t)__reduce_min_sync(kAll, best == top ? who : INT_MAX);
                    sum = b ? sum + key_value(top) : key_value(top);
                }
                if (lane == g) gkey = order_key(sum);
            }
            uint32_t keep = 0;
            for (int b = 0; b < a.top_groups; ++b) {
                const uint32_t top = __reduce_max_sync(kAll, gkey);
                const int g = __ffs(__ballot_sync(kAll, gkey == top)) - 1;
                keep |= 1u << g;
                if (lane == g) gkey = 0;
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = 32 * j + lane;
                if (e < a.E && !((keep >> (e / each)) & 1u)) key[j] = 0;
            }
        }
        int id = 0;  // lane i: the i-th pick
        for (int i = 0; i < a.k; ++i) {
            uint32_t best = 0;
            int who = INT_MAX;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (key[j] > best) best = key[j], who = 32 * j + lane;
            const uint32_t top = __reduce_max_sync(kAll, best);
            const int e = __reduce_min_sync(kAll, best == top ? who : INT_MAX);
            if (lane == i) id = e;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (e == 32 * j + lane) key[j] = 0;
        }
        float w = 0.0f;
        if (lane < a.k) w = score(load_logit(a, at + id));
        if (a.renorm) {
            const float sum = warp_sum(w);
            w = sum == 0.0f ? 0.0f : w / sum;
        }
        if (lane < a.k) {
            a.weights[tok * a.k + lane] = w * a.scale;
            a.ids[tok * a.k + lane] = id;
        }
    }
}

}  // namespace

int launch_route(const void *logits, int64_t ld, const float *bias, float *weights, int32_t *ids, int64_t tokens,
                 int experts, int k, int softmax, int groups, int top_groups, int group_best, int renorm, float scale,
                 int logits_bf16, int num_sms, uint32_t flags, void *stream) {
    RouteArgs a = {logits, bias,       weights,    ids,     tokens, ld,          experts, k,
                   groups, top_groups, group_best, softmax, renorm, logits_bf16, scale};
    const int vpl = (experts + 31) / 32;
    auto fn = vpl <= 1    ? route_kernel<1>
              : vpl <= 2  ? route_kernel<2>
              : vpl <= 4  ? route_kernel<4>
              : vpl <= 8  ? route_kernel<8>
              : vpl <= 16 ? route_kernel<16>
                          : route_kernel<32>;
    const int threads = 128;
    const long long blocks = (tokens + 3) / 4, cap = 16LL * num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
    cfg.blockDim = dim3(threads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace bf16l
