// route.cu — the k experts of each token and their weights from the router's
// logits: softmax or sigmoid scores, a bias for the choice alone, limited groups,
// top-k, renormalised weights.
//
// One warp per token, each lane with a run of VPL neighbouring experts in registers.
// A key is an unsigned word whose order is the float's (NaN and -inf at the bottom, -0
// equal to +0, 0 for an expert that a group limit or an earlier pick took out).  A pick
// is the largest of the lanes' largest keys (one warp reduction) and the first lane
// that has it, which is the lowest expert as runs ascend; a lane keeps its two largest
// keys, so it has to look through its run again only after two picks.  Each group has a
// power of two of lanes to itself and is ranked by a butterfly and a count of the better
// ones; groups too long for that (1023 experts in 3) by reductions over masked keys.
//
// Instructions, not the 1 KB of logits, are the bound of a long batch: a token of 256
// experts takes 1040 with sigmoid, bias, groups and 8 picks, 570 of them up to the keys
// and for the weights, 165 for the groups, 35 to 40 a pick (730 with softmax alone).
// 8192 tokens then are 6.8 us of issue on all SMs, and take 11.0 us (28 with experts
// strided over the lanes and two reductions a pick, 12.6 with one key per lane); softmax
// without groups 7.8.  A short batch is one token's chain: 2.7 us for 1 to 16 tokens of
// 384 and 6 picks, launch included, 3.2 for 1216, 5.1 for 2047 (1.3 of them issue).
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
    int by_logit;     // the logits are the keys
    int vec;          // a lane's run of logits may be read four at a time
    int vec_bias;     // ... and of the bias
    int group_lanes;  // lanes of a group, a power of two; 0 where there are none or a group's run would be too long
    int lane_bits;    // log2 of it
    int each, run;    // experts of a group, and of a lane within it
};

constexpr unsigned kAll = 0xFFFFFFFFu;

// Order-preserving key: a < b as floats <=> key(a) < key(b); -0 as +0; NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float v) {
    v = fmaxf(v, -INFINITY) + 0.0f;  // fmaxf gives the other operand for a NaN
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

// VPL: experts per lane; expert e sits in slot e % VPL of lane e / VPL.
template <int VPL>
__global__ void __launch_bounds__(128) route_kernel(const RouteArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    int e0 = lane * VPL, left = a.E - e0;  // this lane's first expert, and how many there are from it on
    if (a.group_lanes > 0) {
        const int g = lane >> a.lane_bits, at = (lane & (a.group_lanes - 1)) * a.run;
        e0 = g * a.each + at;
        left = g < a.groups ? min(a.run, a.each - at) : 0;
    }
    const long long warps = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long tok = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); tok < a.tokens; tok += warps) {
        const long long at = tok * a.ld;
        float l[VPL];
        if (VPL % 4 == 0 && a.vec) {  // four logits at a time
#pragma unroll
            for (int j = 0; j + 4 <= VPL; j += 4) {
                if (j + 4 > left) {
#pragma unroll
                    for (int i = j; i < j + 4; ++i) l[i] = i < left ? load_logit(a, at + e0 + i) : -INFINITY;
                } else if (a.bf16) {
                    const uint16_t *p = static_cast<const uint16_t *>(a.logits) + at + e0 + j;
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
                    l[j] = bf16_lo(v.x), l[j + 1] = bf16_hi(v.x), l[j + 2] = bf16_lo(v.y), l[j + 3] = bf16_hi(v.y);
                } else {
                    const float *p = static_cast<const float *>(a.logits) + at + e0 + j;
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
                    l[j] = v.x, l[j + 1] = v.y, l[j + 2] = v.z, l[j + 3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) l[j] = j < left ? load_logit(a, at + e0 + j) : -INFINITY;
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
        auto score = [&](float v) {
            if (a.softmax) return total == 0.0f ? 0.0f : expf(v - mx) / total;
            return __frcp_rn(1.0f + expf(-v));  // the quotient, correctly rounded
        };
        uint32_t key[VPL];
        if (a.by_logit) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = j < left ? order_key(l[j]) : 0u;
        } else {
            float b[VPL];
#pragma unroll
            for (int j = 0; j < VPL; ++j) b[j] = 0.0f;
            if (VPL % 4 == 0 && a.bias && a.vec_bias) {
#pragma unroll
                for (int j = 0; j + 4 <= VPL; j += 4) {
                    if (j + 4 > left) {
#pragma unroll
                        for (int i = j; i < j + 4; ++i)
                            if (i < left) b[i] = __ldg(a.bias + e0 + i);
                    } else {
                        const float4 v = __ldg(reinterpret_cast<const float4 *>(a.bias + e0 + j));
                        b[j] = v.x, b[j + 1] = v.y, b[j + 2] = v.z, b[j + 3] = v.w;
                    }
                }
            } else if (a.bias) {
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (j < left) b[j] = __ldg(a.bias + e0 + j);
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const float s = score(l[j]) + b[j];
                key[j] = j < left ? order_key(l[j] == -INFINITY ? l[j] : s) : 0u;
            }
        }
        if (a.group_lanes > 0) {
            // groups of group_lanes lanes: the best two keys of this lane's group, in all its lanes
            uint32_t m1 = 0, m2 = 0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                m2 = max(m2, min(m1, key[j]));
                m1 = max(m1, key[j]);
            }
            for (int o = 1; o < a.group_lanes; o <<= 1) {
                const uint32_t n1 = __shfl_xor_sync(kAll, m1, o), n2 = __shfl_xor_sync(kAll, m2, o);
                m2 = max(min(m1, n1), max(m2, n2));
                m1 = max(m1, n1);
            }
            const uint32_t gkey = order_key(a.group_best == 1 ? key_value(m1) : key_value(m1) + key_value(m2));
            const int mine = lane >> a.lane_bits;
            int better = 0;
            for (int g = 0; g < a.groups; ++g) {
                const uint32_t k = __shfl_sync(kAll, gkey, g << a.lane_bits);
                better += k > gkey || (k == gkey && g < mine);
            }
            if (better >= a.top_groups) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) key[j] = 0;
            }
        } else if (a.groups > 1) {
            const int each = a.each;
            uint32_t gkey = 0;  // lane g: the key of group g
            for (int g = 0; g < a.groups; ++g) {
                const int g0 = g * each - e0, g1 = g0 + each;
                float sum = 0.0f;
                int taken = -1;  // the expert that gave the largest key
                for (int b = 0; b < a.group_best; ++b) {
                    uint32_t best = 0;
                    int who = INT_MAX;
#pragma unroll
                    for (int j = 0; j < VPL; ++j)
                        if (j >= g0 && j < g1 && e0 + j != taken && key[j] > best) best = key[j], who = e0 + j;
                    const uint32_t top = __reduce_max_sync(kAll, best);
                    taken = __reduce_min_sync(kAll, best == top ? who : INT_MAX);
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
            for (int j = 0; j < VPL; ++j)
                if (j < left && !((keep >> ((e0 + j) / each)) & 1u)) key[j] = 0;
        }
        // This lane's largest key and the next, with their slots (equal keys: the lower slot first).
        uint32_t best, next, gone = 0;  // gone: bit j, slot j has been picked
        int slot, slot2, id = 0;        // id, in lane i: the i-th pick
        auto scan = [&] {
            best = gone & 1u ? 0u : key[0], next = 0, slot = 0, slot2 = 0;
#pragma unroll
            for (int j = 1; j < VPL; ++j) {
                const uint32_t k = (gone >> j) & 1u ? 0u : key[j];
                const bool over = k > best, over2 = k > next;
                next = over ? best : over2 ? k : next;
                slot2 = over ? slot : over2 ? j : slot2;
                best = over ? k : best;
                slot = over ? j : slot;
            }
        };
        scan();
        for (int i = 0; i < a.k; ++i) {
            const uint32_t top = __reduce_max_sync(kAll, best);
            const int win = __ffs(__ballot_sync(kAll, best == top)) - 1;
            const int e = __shfl_sync(kAll, e0 + slot, win);
            if (lane == i) id = e;
            if (lane == win) {
                gone |= 1u << slot;
                if (next != 0)  // steps up; its place is filled only if it is picked too
                    best = next, slot = slot2, next = 0;
                else
                    scan();
            }
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
    // Forms by the length of a lane's run, the shortest that is long enough (8192 x 384: 12 12.4 us, 16 19.8).
    static const struct {
        int vpl;
        void (*fn)(const RouteArgs);
    } kForms[] = {{1, route_kernel<1>},   {2, route_kernel<2>},   {3, route_kernel<3>},   {4, route_kernel<4>},
                  {6, route_kernel<6>},   {8, route_kernel<8>},   {12, route_kernel<12>}, {16, route_kernel<16>},
                  {24, route_kernel<24>}, {32, route_kernel<32>}};
    // Each group has a power of two of lanes, unless its runs would be longer than a lane can hold: 7175 x 240 in 16
    // groups 13.6 us (by reductions over masked keys 38.9), 7642 x 272 in 8 12.1 (34.4).
    const int each = experts / groups;
    int group_lanes = 0, lane_bits = 0, run = 0;
    if (groups > 1) {
        while (2 * groups << lane_bits <= 32) ++lane_bits;
        group_lanes = 1 << lane_bits;
        run = (each + group_lanes - 1) / group_lanes;
        if (each % 4 == 0 && run > 3) run = (run + 3) / 4 * 4;  // four at a time
        if (run > 32) group_lanes = 0;
    }
    int form = 0;
    while (kForms[form].vpl < (group_lanes ? run : (experts + 31) / 32)) ++form;
    const int vpl = kForms[form].vpl;
    const bool fours = vpl % 4 == 0 && (group_lanes == 0 || (each % 4 == 0 && run % 4 == 0));
    const uintptr_t bytes = logits_bf16 ? 8 : 16;  // four logits
    RouteArgs a = {logits, bias,       weights,    ids,     tokens, ld,          experts, k,
                   groups, top_groups, group_best, softmax, renorm, logits_bf16, scale};
    a.by_logit = softmax && !bias && group_best == 1;
    a.vec = fours && ld % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % bytes == 0;
    a.vec_bias = fours && (reinterpret_cast<uintptr_t>(bias) & 15u) == 0;
    a.group_lanes = group_lanes;
    a.lane_bits = lane_bits;
    a.each = each;
    a.run = run;
    auto fn = kForms[form].fn;
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
