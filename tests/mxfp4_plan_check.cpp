// Host logic of the MXFP4 split form's plan (csrc/mxfp4_split.cu), without a GPU: one line per plan that is wrong.
#include <stdio.h>

#include <initializer_list>

#include "moe.h"

int main() {
    using namespace bf16l;
    const int Ks[] = {32, 96, 2048, 2880, 4096, 6144, 7168, 65536, 262144}, sms[] = {132, 148, 160};
    int bad = 0;
    for (int K : Ks)
        for (int N = 16; N <= 14336; N += N < 512 ? 16 : 160)
            for (int M : {1, 4, 16, 17, 64})
                for (bool shifted : {false, true}) {
                    const Mxfp4SplitPlan p = mxfp4_split_plan(M, N, K, kGb300Sms, shifted);
                    if (p.smem > 227 * 1024 || p.split < 1 || p.stages < 1) bad += printf("M %d N %d K %d\n", M, N, K);
                    for (int n : sms) {
                        const Mxfp4SplitPlan q = mxfp4_split_plan(M, N, K, n, shifted);
                        if (q.smem > 227 * 1024) bad += printf("M %d N %d K %d on %d SMs: memory\n", M, N, K, n);
                        // codes (planned for the device) and a bf16 x (planned like the workspace) sum in one order
                        if (M <= 16 && (q.split != p.split || q.tokens != p.tokens))
                            bad += printf("M %d N %d K %d on %d SMs: K over %d, on %d over %d\n", M, N, K, n, q.split,
                                          kGb300Sms, p.split);
                    }
                }
    return bad != 0;
}
