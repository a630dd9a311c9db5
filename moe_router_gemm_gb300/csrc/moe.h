// moe.h — internal interface between the C ABI of the operators around the
// linear (api_moe.cu) and their kernels.  Launchers return a cudaError_t value
// (0 on success); arguments have passed the checks of api_moe.cu.
#pragma once

#include "kernels.h"

namespace bf16l {

// As current_device_checked, with the device's kernel status word.  Defined in api.cu.
int current_device_status(bf16l_device *dev, int32_t **status);

// MXFP4 (mxfp4.cu): quantisation and its inverse (n values, n % 32 == 0).
int launch_quant_mxfp4(const void *x, void *q, void *scales, long long n, int num_sms, uint32_t flags, void *stream);
int launch_dequant_mxfp4(const void *q, const void *scales, void *out, long long n, int num_sms, uint32_t flags,
                         void *stream);

// The MXFP4 linear with K over a cluster's CTAs and W on the MMA's M side (mxfp4_split.cu): any M; xs null means that
// x is bf16 and is quantised by the kernel (where mxfp4_split_quantises).
struct Mxfp4SplitPlan {
    int tokens, m_tiles, split, stages;  // tokens and token tiles, CTAs along K, ring depth
    long long smem;                      // dynamic shared memory (more than there is, where a run of x does not fit)
    float estimate;                      // microseconds beside the fixed part, roughly
};
Mxfp4SplitPlan mxfp4_split_plan(int M, int N, int K, int num_sms, bool shifted);
bool mxfp4_split_quantises(int M, int N, int K);
int init_mxfp4_split();
int launch_mxfp4_split(const void *x, const void *xs, const void *wq, const void *ws, const void *bias, void *out,
                       int M, int N, int K, int num_sms, uint32_t flags, void *stream, int32_t *status);
// ... and by CTA pairs on 256 x 256 tiles (mxfp4_pair.cu).
float mxfp4_pair_estimate(int M, int N, int K, int num_sms);  // as Mxfp4SplitPlan::estimate
int init_mxfp4_pair();
int launch_mxfp4_pair(const void *xq, const void *xs, const void *wq, const void *ws, const void *bias, void *out,
                      int M, int N, int K, int num_sms, uint32_t flags, void *stream, int32_t *status);

// Row norm (norm.cu) and routing (route.cu); arguments as in bf16_linear.h.
int launch_rmsnorm(const void *x, int64_t ldx, const void *residual, const void *weight, void *out, void *residual_out,
                   void *codes, void *scales, const float *scale, int64_t rows, int H, float eps, int quant,
                   int num_sms, uint32_t flags, void *stream);
constexpr int kRouteMaxExperts = 1024, kRouteMaxPicks = 32, kRouteMaxGroups = 32;
int launch_route(const void *logits, int64_t ld, const float *bias, float *weights, int32_t *ids, int64_t tokens,
                 int experts, int k, int softmax, int groups, int top_groups, int group_best, int renorm, float scale,
                 int logits_bf16, int num_sms, uint32_t flags, void *stream);

// Rows by group (group.cu): n keys, n + 65536 < 2^31; rest: rows holds the tokens of no group behind the others', where it
// has -1 otherwise.  And a token's rows summed.
constexpr int kMaxGroups = 1024;
int init_group();
int launch_group_rows(const int32_t *ids, int n, int k, int groups, bool rest, int32_t *offsets, int32_t *rows,
                      int32_t *place, uint32_t flags, void *stream);
int launch_combine_rows(const void *y, int64_t y_rows, const int32_t *place, const float *weights, const void *addend,
                        void *out, int64_t tokens, int k, int H, uint32_t flags, void *stream);

// The linear of grouped rows (grouped.cu); N: columns of out, W has 2 N rows a group with swiglu.
struct GroupedArgs {
    const void *x, *w, *bias;
    const int32_t *offsets, *rows;  // rows null: row p of x is row p of out
    void *out;
    int x_rows, P, groups, N, K, swiglu;
    // the adapters' products (launch_lora_*_grouped)
    const float *scale;
    const void *b, *h;
    int R;
    // K in `splits` parts, whose sums go to sums[splits][P][sum_pitch(N)] (of 2 N with swiglu) and are added up after it
    float *sums;
    int splits;
};
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int sum_pitch(int N) { return (N + 7) / 8 * 8; }
int init_grouped();
int grouped_splits(int P, int groups, int N, int K, int swiglu);
int lora_outer_splits(int M, int N, int K);
int launch_grouped(const GroupedArgs &a, int num_sms, uint32_t flags, void *stream, int32_t *status);

// The adapters of a linear.  The inner values h are fp32 sums over `splits` parts of K that are still to be added up and then
// scaled, [splits][M][R], or (splits 0) scaled, [M][2][R] of bf16, first bits and rest.  For rows as they come (lora.cu): the
// inner product, and out from h and the shared product y[M][N] in fp32.  For rows ordered by adapter (grouped.cu, on tensor
// cores): the inner product (splits 0), and out from h, x and w.
constexpr int kLoraMaxRank = 128;
struct LoraArgs {
    const void *x, *a, *b;
    const float *scale;
    const int32_t *ids;
    void *h;
    const float *y;
    void *out;
    int M, N, K, R, L, splits;
    float *sums;  // the shared product's parts, where lora_outer_splits is more than 1
    // y as `parts` parts of K, rows `pitch` apart, still to be added up; `span`: where the inner kernel puts 0 and M
    int parts, pitch;
    int32_t *span;
};
int lora_splits(int M, int K, int R);
int launch_lora_inner(const LoraArgs &a, uint32_t flags, void *stream);
int launch_lora_outer(const LoraArgs &a, uint32_t flags, void *stream);
// ... and for at most kLoraRows rows of at most kLoraRowsSmem bytes in all, the shared product and the adapters' at once.
constexpr int kLoraRows = 2, kLoraRowsSmem = 48 * 1024;
int init_lora();
int launch_lora_rows(const LoraArgs &a, const void *w, const void *bias, uint32_t flags, void *stream);
// The shared product into parts of y (sums), with span as its one group's offsets.
int lora_base_splits(int M, int N, int K);
int launch_lora_base(const LoraArgs &l, const void *w, const void *bias, int num_sms, uint32_t flags, void *stream,
                     int32_t *status);
int launch_lora_inner_grouped(const LoraArgs &l, const int32_t *offsets, const int32_t *rows, int num_sms, uint32_t flags,
                              void *stream, int32_t *status);
int launch_lora_outer_grouped(const LoraArgs &l, const void *w, const void *bias, const int32_t *offsets, const int32_t *rows,
                              int num_sms, uint32_t flags, void *stream, int32_t *status);

}  // namespace bf16l
