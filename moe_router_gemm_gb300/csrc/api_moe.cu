// api_moe.cu — the C ABI of the operators around the linear: norm, routing and
// the 4-bit microscaled form.  As in api.cu, arguments are checked before any
// CUDA call, nothing allocates device memory, nothing synchronises.
#include <stdint.h>

#include "common.cuh"
#include "moe.h"

namespace bf16l {

namespace {

bool off(const void *p, uintptr_t align) { return (reinterpret_cast<uintptr_t>(p) & (align - 1)) != 0; }

struct Span {
    const void *p;
    uint64_t bytes;
};

bool meet(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// No output overlaps an input or another output.
template <int NO, int NI>
bool clash(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(outs[i], ins[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (meet(outs[i], outs[j])) return true;
    }
    return false;
}

int result(int cuda_err) {
    if (!cuda_err) return BF16L_OK;
    note_cuda_error(cuda_err);
    return BF16L_ELAUNCH;
}

constexpr uint64_t kMaxElements = 1ull << 40;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Checks of the MXFP4 product that need no GPU, but the pointers of x.
int check_linear(const void *wq, const void *ws, const void *bias, const void *out, int M, int N, int K,
                 uint32_t flags) {
    if (M < 0 || N <= 0 || K <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (K % 32 != 0) return BF16L_EUNSUPPORTED;
    if (M == 0) return BF16L_OK;
    if (!wq || !ws || !out) return BF16L_EINVAL;
    if (off(wq, 16) || off(out, 16) || (bias && off(bias, 16))) return BF16L_EALIGN;
    if ((uint64_t)M * (uint64_t)N > kMaxElements) return BF16L_EINVAL;
    return BF16L_OK;
}

}  // namespace

}  // namespace bf16l

using namespace bf16l;

extern "C" int bf16_rmsnorm(const void *x, int64_t ldx, const void *residual, const void *weight, void *out,
                            void *residual_out, void *codes, void *scales, const float *scale, int64_t rows, int H,
                            float eps, int quant, uint32_t flags, bf16l_stream_t stream) {
    if (rows < 0 || H <= 0 || ldx < H || !flags_valid(flags)) return BF16L_EINVAL;
    if (quant < BF16L_QUANT_NONE || quant > BF16L_QUANT_MXFP4) return BF16L_EINVAL;
    if (!(eps >= 0.0f)) return BF16L_EINVAL;
    const bool mx = quant == BF16L_QUANT_MXFP8 || quant == BF16L_QUANT_MXFP4;
    if (mx && H % 32 != 0) return BF16L_EUNSUPPORTED;
    if (rows == 0) return BF16L_OK;
    if (!x || !weight || (residual != nullptr) != (residual_out != nullptr)) return BF16L_EINVAL;
    if ((uint64_t)rows > kMaxElements / (uint64_t)ldx) return BF16L_EINVAL;
    if (quant == BF16L_QUANT_NONE ? !out : (!codes || (mx ? !scales : !scale))) return BF16L_EINVAL;
    if (off(x, 2) || off(weight, 16) || off(residual, 16) || off(residual_out, 16) || off(out, 16)) return BF16L_EALIGN;
    if (quant != BF16L_QUANT_NONE && off(codes, 16)) return BF16L_EALIGN;
    if (quant == BF16L_QUANT_FP8 && off(scale, 4)) return BF16L_EALIGN;
    const uint64_t n = (uint64_t)rows * (uint64_t)H;
    const Span outs[4] = {{out, 2 * n},
                          {residual_out, 2 * n},
                          {quant ? codes : nullptr, quant == BF16L_QUANT_MXFP4 ? n / 2 : n},
                          {mx ? scales : nullptr, n / 32}};
    const Span ins[4] = {{x, 2 * ((uint64_t)(rows - 1) * (uint64_t)ldx + (uint64_t)H)},
                         {weight, 2ull * (uint64_t)H},
                         {residual == residual_out ? nullptr : residual, 2 * n},
                         {quant == BF16L_QUANT_FP8 ? scale : nullptr, 4}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_rmsnorm(x, ldx, residual, weight, out, residual_out, codes, scales, scale, rows, H, eps, quant,
                                 dev.num_sms, flags, stream));
}

extern "C" int bf16_route(const void *logits, int64_t ld, const float *bias, float *weights, int32_t *ids,
                          int64_t tokens, int experts, int k, int scoring, int groups, int top_groups, int group_best,
                          int renormalize, float scale, int logits_bf16, uint32_t flags, bf16l_stream_t stream) {
    if (tokens < 0 || experts <= 0 || ld < experts || k <= 0 || groups <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (scoring != BF16L_SCORE_SOFTMAX && scoring != BF16L_SCORE_SIGMOID) return BF16L_EINVAL;
    if (experts > kRouteMaxExperts || k > kRouteMaxPicks || groups > kRouteMaxGroups) return BF16L_EUNSUPPORTED;
    if (experts % groups != 0 || top_groups < 1 || top_groups > groups) return BF16L_EINVAL;
    const int each = experts / groups;
    if (group_best < 1 || group_best > 2 || group_best > each || k > top_groups * each) return BF16L_EINVAL;
    if (tokens == 0) return BF16L_OK;
    if (!logits || !weights || !ids) return BF16L_EINVAL;
    if ((uint64_t)tokens > kMaxElements / (uint64_t)ld) return BF16L_EINVAL;
    const uint64_t el = logits_bf16 ? 2 : 4;
    if (off(logits, el) || off(weights, 4) || off(ids, 4) || off(bias, 4)) return BF16L_EALIGN;
    const Span outs[2] = {{weights, 4ull * (uint64_t)tokens * k}, {ids, 4ull * (uint64_t)tokens * k}};
    const Span ins[2] = {{logits, el * ((uint64_t)(tokens - 1) * (uint64_t)ld + (uint64_t)experts)},
                         {bias, 4ull * (uint64_t)experts}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_route(logits, ld, bias, weights, ids, tokens, experts, k, scoring == BF16L_SCORE_SOFTMAX,
                               groups, top_groups, group_best, renormalize != 0, scale, logits_bf16 != 0, dev.num_sms,
                               flags, stream));
}

extern "C" int bf16_quant_mxfp4(const void *x, int64_t rows, int K, void *xq, void *xs, uint32_t flags,
                                bf16l_stream_t stream) {
    if (rows < 0 || K <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (K % 32 != 0) return BF16L_EUNSUPPORTED;
    if (rows == 0) return BF16L_OK;
    if (!x || !xq || !xs) return BF16L_EINVAL;
    if (off(x, 16) || off(xq, 16)) return BF16L_EALIGN;
    if ((uint64_t)rows > kMaxElements / (uint64_t)K) return BF16L_EINVAL;
    const uint64_t n = (uint64_t)rows * (uint64_t)K;
    const Span outs[2] = {{xq, n / 2}, {xs, n / 32}}, ins[1] = {{x, 2 * n}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_quant_mxfp4(x, xq, xs, (long long)n, dev.num_sms, flags, stream));
}

extern "C" int bf16_dequant_mxfp4(const void *xq, const void *xs, int64_t rows, int K, void *out, uint32_t flags,
                                  bf16l_stream_t stream) {
    if (rows < 0 || K <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (K % 32 != 0) return BF16L_EUNSUPPORTED;
    if (rows == 0) return BF16L_OK;
    if (!xq || !xs || !out) return BF16L_EINVAL;
    if (off(xq, 16) || off(out, 16)) return BF16L_EALIGN;
    if ((uint64_t)rows > kMaxElements / (uint64_t)K) return BF16L_EINVAL;
    const uint64_t n = (uint64_t)rows * (uint64_t)K;
    const Span outs[1] = {{out, 2 * n}}, ins[2] = {{xq, n / 2}, {xs, n / 32}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_dequant_mxfp4(xq, xs, out, (long long)n, dev.num_sms, flags, stream));
}

extern "C" int bf16_linear_mxfp4(const void *xq, const void *xs, const void *wq, const void *ws, const void *bias,
                                 void *out, int M, int N, int K, uint32_t flags, bf16l_stream_t stream) {
    int st = check_linear(wq, ws, bias, out, M, N, K, flags);
    if (st != BF16L_OK || M == 0) return st;
    if (!xq || !xs) return BF16L_EINVAL;
    if (off(xq, 16)) return BF16L_EALIGN;
    const uint64_t m = (uint64_t)M, n = (uint64_t)N, k = (uint64_t)K;
    const Span outs[1] = {{out, 2 * m * n}};
    const Span ins[5] = {{xq, m * k / 2}, {xs, m * k / 32}, {wq, n * k / 2}, {ws, n * k / 32}, {bias, 2 * n}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    int32_t *status = nullptr;
    st = current_device_status(&dev, &status);
    if (st != BF16L_OK) return st;
    // Few tokens, or few tiles for their K: the split form.  512 x 2112 x 7168: split 14.4 us, pairs 15.4; 1024 x 2112 x
    // 7168: 21.9 and 15.1; 1000 x 256 x 7168: 8.0 and 13.7; 128 x 14336 x 4096: 15.3 and 11.3.
    if (M > 16 &&
        mxfp4_pair_estimate(M, N, K, dev.num_sms) < mxfp4_split_plan(M, N, K, dev.num_sms, false).estimate)
        return result(launch_mxfp4_pair(xq, xs, wq, ws, bias, out, M, N, K, dev.num_sms, flags, stream, status));
    return result(launch_mxfp4_split(xq, xs, wq, ws, bias, out, M, N, K, dev.num_sms, flags, stream, status));
}

extern "C" size_t bf16_linear_mxfp4_dynamic_workspace(int M, int N, int K) {
    if (M <= 0 || N <= 0 || K <= 0 || K % 32 != 0) return 0;
    if (mxfp4_split_quantises(M, N, K)) return 0;
    return up256((size_t)M * (size_t)(K / 2)) + up256((size_t)M * (size_t)(K / 32));
}

extern "C" int bf16_linear_mxfp4_dynamic(const void *x, const void *wq, const void *ws, const void *bias, void *out,
                                         int M, int N, int K, void *workspace, size_t workspace_bytes, uint32_t flags,
                                         bf16l_stream_t stream) {
    int st = check_linear(wq, ws, bias, out, M, N, K, flags);
    if (st != BF16L_OK || M == 0) return st;
    if (!x) return BF16L_EINVAL;
    if (off(x, 16) || (workspace && off(workspace, 256))) return BF16L_EALIGN;
    const size_t need = bf16_linear_mxfp4_dynamic_workspace(M, N, K);
    if (need && (!workspace || workspace_bytes < need)) return BF16L_EINVAL;
    const uint64_t m = (uint64_t)M, n = (uint64_t)N, k = (uint64_t)K;
    const Span outs[2] = {{out, 2 * m * n}, {workspace, need}};
    const Span ins[4] = {{x, 2 * m * k}, {wq, n * k / 2}, {ws, n * k / 32}, {bias, 2 * n}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    if (need == 0) {  // the kernel quantises x itself
        bf16l_device dev;
        int32_t *status = nullptr;
        st = current_device_status(&dev, &status);
        if (st != BF16L_OK) return st;
        return result(launch_mxfp4_split(x, nullptr, wq, ws, bias, out, M, N, K, dev.num_sms, flags, stream, status));
    }
    uint8_t *xq = static_cast<uint8_t *>(workspace);
    uint8_t *xs = xq + up256((size_t)M * (size_t)(K / 2));
    st = bf16_quant_mxfp4(x, M, K, xq, xs, flags, stream);
    if (st != BF16L_OK) return st;
    return bf16_linear_mxfp4(xq, xs, wq, ws, bias, out, M, N, K, flags, stream);
}
