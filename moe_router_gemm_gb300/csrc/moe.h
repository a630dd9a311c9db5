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

}  // namespace bf16l
