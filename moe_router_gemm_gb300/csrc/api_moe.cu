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
constexpr int64_t kMaxRows = 0x7FFFFFFF - 65536;  // rows of a group's matrix, so that a tile past the last fits an int
constexpr int kMaxWidth = 1 << 24;                // ... and their length

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

extern "C" int bf16_group_rows(const int32_t *ids, int64_t tokens, int k, int groups, int32_t *offsets, int32_t *rows,
                               int32_t *place, uint32_t flags, bf16l_stream_t stream) {
    if (tokens < 0 || k <= 0 || groups <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (groups > kMaxGroups) return BF16L_EUNSUPPORTED;
    if (tokens > kMaxRows / k) return BF16L_EINVAL;
    const uint64_t n = (uint64_t)tokens * (uint64_t)k;
    if (!offsets || (n && (!ids || !rows))) return BF16L_EINVAL;
    if (off(ids, 4) || off(offsets, 4) || off(rows, 4) || off(place, 4)) return BF16L_EALIGN;
    const Span outs[3] = {{offsets, 4ull * ((uint64_t)groups + 1)}, {rows, 4 * n}, {place, 4 * n}};
    const Span ins[1] = {{ids, 4 * n}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_group_rows(ids, (int)n, k, groups, false, offsets, rows, place, flags, stream));
}

namespace {

// What the call and its workspace's size refuse alike.
int check_grouped_sizes(int64_t P, int groups, int N, int K, int swiglu) {
    if (P < 0 || groups <= 0 || N <= 0 || K <= 0) return BF16L_EINVAL;
    if (K % 8 != 0 || groups > kMaxGroups || N > kMaxWidth || K > kMaxWidth) return BF16L_EUNSUPPORTED;
    if (P > kMaxRows) return BF16L_EINVAL;
    if (P == 0) return BF16L_OK;
    const uint64_t wide = (uint64_t)N * (swiglu ? 2 : 1);
    return (uint64_t)P * wide > kMaxElements || (uint64_t)groups * wide > kMaxElements / (uint64_t)K ? BF16L_EINVAL : BF16L_OK;
}

}  // namespace

extern "C" size_t bf16_linear_grouped_workspace(int64_t P, int groups, int N, int K, int swiglu) {
    if (P == 0 || check_grouped_sizes(P, groups, N, K, swiglu) != BF16L_OK) return 0;
    const int s = grouped_splits((int)P, groups, N, K, swiglu);
    return s > 1 ? up256(4 * (size_t)s * (size_t)P * (size_t)sum_pitch(swiglu ? 2 * N : N)) : 0;
}

extern "C" int bf16_linear_grouped(const void *x, int64_t x_rows, const void *w, const void *bias, const int32_t *offsets,
                                   const int32_t *rows, void *out, int64_t P, int groups, int N, int K, int swiglu,
                                   void *workspace, size_t workspace_bytes, uint32_t flags, bf16l_stream_t stream) {
    if (x_rows < 0 || !flags_valid(flags)) return BF16L_EINVAL;
    int st = check_grouped_sizes(P, groups, N, K, swiglu);
    if (st != BF16L_OK) return st;
    if (x_rows > kMaxRows) return BF16L_EINVAL;
    if (P == 0) return BF16L_OK;  // (an empty `rows` may be NULL)
    if (!rows && x_rows != P) return BF16L_EINVAL;
    if (!x || !w || !offsets || !out || x_rows == 0) return BF16L_EINVAL;
    if (off(x, 16) || off(w, 16) || off(bias, 16) || off(out, 16) || off(offsets, 4) || off(rows, 4)) return BF16L_EALIGN;
    const uint64_t k = (uint64_t)K, wide = (uint64_t)N * (swiglu ? 2 : 1), g = (uint64_t)groups;
    const size_t need = bf16_linear_grouped_workspace(P, groups, N, K, swiglu);
    if (off(workspace, 256)) return BF16L_EALIGN;
    if (need && (!workspace || workspace_bytes < need)) return BF16L_EINVAL;
    const Span outs[2] = {{out, 2ull * (uint64_t)P * (uint64_t)N}, {workspace, need}};
    const Span ins[5] = {{x, 2ull * (uint64_t)x_rows * k}, {w, 2 * g * wide * k}, {bias, 2 * g * wide},
                         {offsets, 4 * (g + 1)}, {rows, 4ull * (uint64_t)P}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    int32_t *status = nullptr;
    st = current_device_status(&dev, &status);
    if (st != BF16L_OK) return st;
    const GroupedArgs a = {x, w, bias, offsets, rows, out, (int)x_rows, (int)P, groups, N, K, swiglu != 0, nullptr, nullptr,
                           nullptr, 0, static_cast<float *>(workspace), need ? grouped_splits((int)P, groups, N, K, swiglu) : 1};
    return result(launch_grouped(a, dev.num_sms, flags, stream, status));
}

extern "C" int bf16_combine_rows(const void *y, int64_t y_rows, const int32_t *place, const float *weights,
                                 const void *addend, void *out, int64_t tokens, int k, int H, uint32_t flags,
                                 bf16l_stream_t stream) {
    if (tokens < 0 || y_rows < 0 || k <= 0 || H <= 0 || !flags_valid(flags)) return BF16L_EINVAL;
    if (tokens == 0) return BF16L_OK;
    if ((y_rows && !y) || !place || !out) return BF16L_EINVAL;
    if (off(y, 16) || off(addend, 16) || off(out, 16) || off(place, 4) || off(weights, 4)) return BF16L_EALIGN;
    const uint64_t h = (uint64_t)H, t = (uint64_t)tokens;
    if (t > kMaxElements / h || (uint64_t)y_rows > kMaxElements / h || t > kMaxElements / (uint64_t)k) return BF16L_EINVAL;
    const Span outs[1] = {{out, 2 * t * h}};
    const Span ins[4] = {{y, 2ull * (uint64_t)y_rows * h}, {place, 4 * t * (uint64_t)k}, {weights, 4 * t * (uint64_t)k},
                         {addend == out ? nullptr : addend, 2 * t * h}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    const int st = current_device_checked(&dev);
    if (st != BF16L_OK) return st;
    return result(launch_combine_rows(y, y_rows, place, weights, addend, out, tokens, k, H, flags, stream));
}

namespace {

// What the call and its workspace's size refuse alike.
int check_lora_sizes(int M, int N, int K, int R, int L) {
    if (M < 0 || N <= 0 || K <= 0 || R <= 0 || L <= 0) return BF16L_EINVAL;
    if (K % 8 != 0 || R % 8 != 0 || R > kLoraMaxRank || L > kMaxGroups || N > kMaxWidth || K > kMaxWidth)
        return BF16L_EUNSUPPORTED;
    if (M == 0) return BF16L_OK;
    const uint64_t adapters = (uint64_t)L * (uint64_t)R * (uint64_t)(N > K ? N : K);
    return M > kMaxRows || (uint64_t)M * (uint64_t)N > kMaxElements || adapters > kMaxElements ? BF16L_EINVAL : BF16L_OK;
}

// How a linear with adapters is done, by sizes alone, and the parts of its workspace.
//   cores: the inner products row by row on CUDA cores, each row reading its own adapter from L2, or rows in adapter order
//     on tensor cores, by estimate: (1.5 + K / 1400) us for each 1824 blocks of four ranks of a row, 6 + K / 320 us.
//     (Whole calls, us: 435 x 377 x 5944 with rank 32 34.9 and 42.0, 2000 x 512 x 512 with rank 64 44.7 and 21.6.)
//   fused: the shared product and the adapters' by one tensor-core kernel on tiles of 256 rows; for few rows the dense
//     linear's own kernels, which split K, into fp32 and the adapters' share after it (61 x 2112 x 7168 with rank 32: 18 us,
//     30 fused; 281 x 322 x 2880 with rank 32: 43 and 24).
//   parted: between the two, the grouped linear's kernel with the rows on its N side, into fp32 parts, and the adapters' share
//     after it, for which every row reads its own B: up to kPartedRows rows and kPartedWork of M N R (us, fused in brackets:
//     65 x 4096 x 4096 r16 21.0 (28.8), 128 x 4096 x 4096 r16 25.2 (34.0), 96 x 2112 x 7168 r32 27.8 (35.2), 128 x 2048 x 7168
//     r64 35.0 (37.5); past the bounds 128 x 14336 x 4096 r16 43.8 (41.7), 256 x 4096 x 4096 r16 34.7 (33.8)).
constexpr int kPartedRows = 160;
constexpr uint64_t kPartedWork = 20ull << 20;
struct LoraWay {
    bool cores, fused, parted;
    int parts, pitch;
    size_t order, h, y;  // bytes: the rows' order, the inner values, the shared product or its parts
};
LoraWay lora_way(int M, int N, int K, int R, int L) {
    const uint64_t m = (uint64_t)M, r = (uint64_t)R;
    LoraWay w;
    w.parted = M > 64 && M <= kPartedRows && m * r * (uint64_t)N <= kPartedWork;
    w.fused = M > 64 && !w.parted;
    w.cores = !w.fused || m * r / 4 * (2100 + (uint64_t)K) * 320 <= 1824ull * 1400 * (1920 + (uint64_t)K);
    w.order = w.fused ? up256(4 * ((size_t)L + 1)) + up256(4 * m) : w.parted ? 256 : 0;
    w.h = up256((w.fused ? 1 : (size_t)lora_splits(M, K, R)) * 4 * m * r);
    w.parts = w.fused ? lora_outer_splits(M, N, K) : w.parted ? lora_base_splits(M, N, K) : 1;
    w.pitch = w.parted || w.parts > 1 ? sum_pitch(N) : N;
    w.y = w.fused && w.parts == 1 ? 0 : up256((size_t)w.parts * 4 * m * (size_t)w.pitch);
    return w;
}

// The dense linear's plan for few rows, where its table has no line for most sizes: the forms that lead there, by the fill of
// the SMs (fp32 out, us; the general rule in brackets): 8 x 4096 x 4096 6.6 (22.2), 8 x 7168 x 2048 6.2 (22.2), 16 x 4096 x
// 4096 7.8 (11.7), 32 x 4096 x 4096 10.4 (12.4), 61 x 2112 x 7168 10.9 (15.5), 64 x 7168 x 7168 24.2 (28.2).  Narrow weights
// stay with the general rule.  One row comes here with K past 24576 alone (lora_rows): 1 x 1024 x 26000 15.4 (14.1), 1 x 2048 x
// 26000 16.7 (21.6), 1 x 4096 x 26000 30.4 (42.8).
bool few_rows_plan(int M, int N, int K, const bf16l_device &dev, uint32_t flags, bf16l_plan *plan) {
    bf16l_plan p = {};
    p.flags = (int32_t)flags;
    if (N < (M == 1 ? 2048 : 1024) || M > 64 || (M > 16 && N > 8192)) return false;  // (64 x 14336 x 4096: 24.9, 31 so)
    if (M <= 16) {  // 16 W rows for some warps of 16 an SM, all of them at work
        p.kernel = BF16L_KERNEL_WARPMMA;
        p.threads = 512;
        p.tokens_per_cta = 2;
        p.split_k = 1;
        p.stages = 1;
        p.rows_per_cta = 4;
        while (p.rows_per_cta < 16 && 2 * p.rows_per_cta * ((N + 15) / 16) <= 18 * dev.num_sms) p.rows_per_cta *= 2;
    } else {  // K over a cluster, two CTAs an SM
        p.kernel = BF16L_KERNEL_SPLITK;
        p.threads = kSplitThreads;
        p.rows_per_cta = N < 6144 ? 64 : 96;
        p.tokens_per_cta = (M + 7) / 8 * 8;
        p.stages = 2;
        p.chunks_per_stage = 2;
        const int tiles = (N + p.rows_per_cta - 1) / p.rows_per_cta, most = (K + 2 * kChunkK - 1) / (2 * kChunkK);
        p.split_k = (2 * dev.num_sms - tiles / 2) / tiles;
        p.split_k = p.split_k < 1 ? 1 : p.split_k > 8 ? 8 : p.split_k;
        if (p.split_k > most) p.split_k = most;
    }
    *plan = p;
    return check_plan(M, N, K, dev, &p) == BF16L_OK;
}

}  // namespace

extern "C" size_t bf16_linear_lora_workspace(int M, int N, int K, int R, int L) {
    if (M == 0 || check_lora_sizes(M, N, K, R, L) != BF16L_OK) return 0;
    const LoraWay w = lora_way(M, N, K, R, L);
    return w.order + w.h + w.y;
}

extern "C" int bf16_linear_lora(const void *x, const void *w, const void *bias, const void *a, const void *b,
                                const float *scale, const int32_t *ids, void *out, int M, int N, int K, int R, int L,
                                void *workspace, size_t workspace_bytes, uint32_t flags, bf16l_stream_t stream) {
    if (!flags_valid(flags)) return BF16L_EINVAL;
    int st = check_lora_sizes(M, N, K, R, L);
    if (st != BF16L_OK || M == 0) return st;
    if (!x || !w || !a || !b || !ids || !out) return BF16L_EINVAL;
    if (off(x, 16) || off(w, 16) || off(bias, 16) || off(a, 16) || off(b, 16) || off(out, 16) || off(scale, 4) ||
        off(ids, 4) || off(workspace, 256))
        return BF16L_EALIGN;
    const uint64_t m = (uint64_t)M, n = (uint64_t)N, k = (uint64_t)K, r = (uint64_t)R, l = (uint64_t)L;
    const size_t need = bf16_linear_lora_workspace(M, N, K, R, L);
    if (!workspace || workspace_bytes < need) return BF16L_EINVAL;
    const Span outs[2] = {{out, 2 * m * n}, {workspace, need}};
    const Span ins[7] = {{x, 2 * m * k}, {w, 2 * n * k}, {bias, 2 * n}, {a, 2 * l * r * k}, {b, 2 * l * r * n},
                         {scale, 4 * l}, {ids, 4 * m}};
    if (clash(outs, ins)) return BF16L_EINVAL;
    bf16l_device dev;
    int32_t *status = nullptr;
    st = current_device_status(&dev, &status);
    if (st != BF16L_OK) return st;
    const LoraWay way = lora_way(M, N, K, R, L);
    uint8_t *p = static_cast<uint8_t *>(workspace);
    int32_t *offsets = reinterpret_cast<int32_t *>(p), *rows = reinterpret_cast<int32_t *>(p + up256(4 * ((size_t)L + 1)));
    float *y = reinterpret_cast<float *>(p + way.order + way.h);
    const LoraArgs args = {x, a, b, scale, ids, p + way.order, y, out, M, N, K, R, L,
                           way.fused ? 0 : lora_splits(M, K, R), y,
                           way.parts, way.pitch, way.parted ? offsets : nullptr};
    if (way.fused) st = result(launch_group_rows(ids, M, 1, L, true, offsets, rows, nullptr, flags, stream));
    if (st == BF16L_OK)
        st = result(way.cores ? launch_lora_inner(args, flags, stream)
                              : launch_lora_inner_grouped(args, offsets, rows, dev.num_sms, flags, stream, status));
    if (st != BF16L_OK) return st;
    if (way.fused)
        return result(launch_lora_outer_grouped(args, w, bias, offsets, rows, dev.num_sms, flags, stream, status));
    if (M <= kLoraRows && (int64_t)M * K * 2 <= kLoraRowsSmem)  // (few rows: cores, with splits)
        return result(launch_lora_rows(args, w, bias, flags, stream));
    if (way.parted) {
        st = result(launch_lora_base(args, w, bias, dev.num_sms, flags, stream, status));
        return st != BF16L_OK ? st : result(launch_lora_outer(args, flags, stream));
    }
    // The product may read its weights as soon as the inner kernel lets it start: that one has waited for all before it.
    bf16l_plan plan;
    const uint32_t early = flags & BF16L_FLAG_SERIAL ? flags : flags | BF16L_FLAG_PDL;
    st = few_rows_plan(M, N, K, dev, early, &plan) ? bf16_linear_f32out_with_plan(x, w, bias, y, M, N, K, &plan, stream)
                                                   : bf16_linear_f32out(x, w, bias, y, M, N, K, early, stream);
    return st != BF16L_OK ? st : result(launch_lora_outer(args, flags, stream));
}
