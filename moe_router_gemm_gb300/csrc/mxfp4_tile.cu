// mxfp4_tile.cu — the MXFP4 linear for many tokens: tcgen05.mma.kind::mxf4.block_scale,
// two 32-code scale blocks per instruction, scales applied by the tensor core.
//
//   * tile 128 x rows (MMA M) x BQ W rows (MMA N, 128 or 256); a stage is one
//     256-code chunk of both operands (128-byte swizzle rows, TMA) = eight scale
//     blocks = four MMAs;
//   * warp 0 loads the codes (TMA), warp 1 issues the MMAs and owns TMEM, warps
//     2-5 run the epilogue (TMEM lane = x row; bias, bf16 store), warps 6-9 stage
//     each chunk's scale words into TMEM ahead of the MMAs: words 0 and 1 of row r
//     for chunk c are the bytes xs[r][8c..8c+3] and xs[r][8c+4..8c+7], and MMA kk
//     reads bytes 2(kk % 2) and 2(kk % 2) + 1 of word kk / 2 (the descriptor's
//     scale id);
//   * TMEM: the accumulator (two BQ-column buffers for BQ = 128, one for 256, whose
//     epilogue then runs between tiles), then 32 columns of scales per ring stage:
//     A word 0 at 0, A word 1 at 8, B word 0 at 16, B word 1 at 24 (every address a
//     multiple of 8).  A row m's word sits in lane m of column m / 32, B row n's in
//     lane n % 32 of column n / 32 of every lane quarter;
//   * K past its end: the codes are zero (TMA fill) and the scale bytes 1.0.
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

constexpr int kBP = 128, kChunkBytes = 128;
constexpr int kMaxStages = 7;
constexpr int kSlot = 32;

__host__ __device__ constexpr int stage_bytes(int bq) { return (kBP + bq) * kChunkBytes; }

struct TileShared {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t sfull[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem_base;
    int32_t aborted;
    int32_t issued;
    int32_t consumed;
};

__device__ __forceinline__ void fp4_coords(int t, int p_tiles, int q_tiles, int group, int bq, int &p0, int &q0) {
    const int per_group = group * p_tiles;
    const int g = t / per_group, r = t - g * per_group;
    const int gq = (q_tiles - g * group) < group ? (q_tiles - g * group) : group;
    const int pi = r / gq, qi = g * group + (r - pi * gq);
    p0 = pi * kBP;
    q0 = qi * bq;
}

// The scale words of chunk c of one row (nb bytes): bytes 8c..8c+7, those past nb read as 1.0.
// W: bytes the row's start and length are multiples of (8, 4 or 1).
template <int W>
__device__ __forceinline__ uint2 scale_words(const uint8_t *row, int c, int nb, bool in) {
    uint2 v = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const int b = 8 * c;
    if (!in || b >= nb) return v;
    if (W == 8) return __ldg(reinterpret_cast<const uint2 *>(row + b));
    if (W == 4) {
        v.x = __ldg(reinterpret_cast<const uint32_t *>(row + b));
        if (b + 4 < nb) v.y = __ldg(reinterpret_cast<const uint32_t *>(row + b + 4));
        return v;
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= (uint32_t)(b + i < nb ? __ldg(row + b + i) : 0x7F) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

template <int BQ, int W>
__global__ void __launch_bounds__(kMxfp4TileThreads, 1)
    mxfp4_tile_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const uint8_t *__restrict__ xs, const uint8_t *__restrict__ ws,
                      const uint16_t *__restrict__ bias, uint16_t *__restrict__ out, int M, int N, int K, int stages,
                      int group, int32_t *status) {
    constexpr int kNbuf = BQ == 128 ? 2 : 1;  // accumulator buffers
    constexpr int kBcols = BQ / 32;           // B scale columns per word
    constexpr int kSf = kNbuf * BQ;           // the scale slots start after the accumulators
    constexpr int kStageBytes = stage_bytes(BQ);
    static_assert(kSf + kMaxStages * kSlot <= 512, "TMEM columns");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    TileShared &sh = *reinterpret_cast<TileShared *>(ring + stages * kStageBytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int p_tiles = (M + kBP - 1) / kBP, q_tiles = (N + BQ - 1) / BQ;
    const int num_tiles = p_tiles * q_tiles;
    const int C = (K + 2 * kChunkBytes - 1) / (2 * kChunkBytes);
    const int nb = K >> 5;  // scale bytes per row

    if (tid == 0) {
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
            mbar_init(&sh.sfull[s], 4);  // one arrival per scale warp
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], 4);  // one arrival per epilogue warp
        }
        sh.aborted = 0;
        sh.issued = 0;
        sh.consumed = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    pdl_launch_dependents();
    pdl_wait();  // nothing is read before the previous kernel has finished

    if (warp == 0) {
        if (lane == 0) {  // ---- TMA producer: the codes ----
            int it = 0;
            for (int t = blockIdx.x; t < num_tiles; t += gridDim.x) {
                int p0, q0;
                fp4_coords(t, p_tiles, q_tiles, group, BQ, p0, q0);
                for (int c = 0; c < C; ++c, ++it) {
                    const int s = it % stages;
                    if (it >= stages && !mbar_wait(&sh.empty[s], ((it / stages) - 1) & 1, status, kSiteEmpty)) {
                        atomicExch(&sh.aborted, 1);
                        goto producer_done;
                    }
                    if (*((volatile int32_t *)&sh.aborted)) goto producer_done;
                    uint8_t *st = ring + s * kStageBytes;
                    mbar_arrive_expect_tx(&sh.full[s], kStageBytes);
                    tma_load_2d(st, &tm_x, &sh.full[s], c * kChunkBytes, p0);
                    tma_load_2d(st + kBP * kChunkBytes, &tm_w, &sh.full[s], c * kChunkBytes, q0);
                }
            }
        producer_done:
            sh.issued = it;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {  // ---- MMA issuer ----
            int it = 0, tile_iter = 0;
            for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++tile_iter) {
                sh.consumed = it;
                const int b = tile_iter % kNbuf, use = tile_iter / kNbuf;
                const uint32_t acc = tmem + (uint32_t)(b * BQ);
                // wait for the epilogue to have drained this buffer (its previous use)
                if (use >= 1 && !mbar_wait(&sh.acc_empty[b], (use - 1) & 1, status, kSiteTmemEmpty)) {
                    atomicExch(&sh.aborted, 1);
                    break;
                }
                tc_fence_after();
                bool ok = true;
                for (int c = 0; c < C; ++c, ++it) {
                    const int s = it % stages;
                    if (!mbar_wait(&sh.full[s], (it / stages) & 1, status, kSiteFull) ||
                        !mbar_wait(&sh.sfull[s], (it / stages) & 1, status, kSiteFull)) {
                        atomicExch(&sh.aborted, 1);
                        sh.consumed = it;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *st = ring + s * kStageBytes;
                    const uint64_t adesc = smem_desc_sw128(smem_u32(st));
                    const uint64_t bdesc = smem_desc_sw128(smem_u32(st + kBP * kChunkBytes));
                    const uint32_t sf = tmem + (uint32_t)(kSf + kSlot * s);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 64 codes, two scale blocks
                        mma_mxf4(acc, adesc + 2 * kk, bdesc + 2 * kk, idesc_mxf4_f32(kBP, BQ, 2 * (kk & 1)),
                                 sf + 8 * (kk >> 1), sf + 16 + 8 * (kk >> 1), (c > 0 || kk > 0) ? 1u : 0u);
                    mma_commit(&sh.empty[s]);  // frees the codes and the scale slot
                }
                if (!ok) {
                    mbar_arrive(&sh.acc_full[b]);
                    break;
                }
                mma_commit(&sh.acc_full[b]);
            }
            sh.consumed = it;
        }
        __syncwarp();
    } else if (warp < 6) {
        // ---- epilogue: warps 2..5; TMEM lane quarter = warp % 4 ----
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        int tile_iter = 0;
        const bool vec_ok = (N % 8) == 0;
        for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++tile_iter) {
            int p0, q0;
            fp4_coords(t, p_tiles, q_tiles, group, BQ, p0, q0);
            const int b = tile_iter % kNbuf, use = tile_iter / kNbuf;
            // The tile's bias, one value per lane and 32-column slice, read while the MMAs run.
            float lbs[BQ / 32];
#pragma unroll
            for (int i = 0; i < BQ / 32; ++i) lbs[i] = bias_lane(bias, q0 + 32 * i, N);
            const bool ok = mbar_wait(&sh.acc_full[b], use & 1, status, kSiteAccum);
            tc_fence_after();
            // warp-uniform, so that the bias shuffles below run on all 32 lanes
            const bool have = __all_sync(0xFFFFFFFFu, ok && !*((volatile int32_t *)&sh.aborted));
            const int m = p0 + row;
            const uint32_t acc = tmem + (uint32_t)(b * BQ) + ((uint32_t)(quarter * 32) << 16);
            if (have) {
#pragma unroll
                for (int c = 0; c < BQ; c += 32) {
                    uint32_t r0[16], r1[16];
                    tmem_ld16(acc + (uint32_t)c, r0);
                    tmem_ld16(acc + (uint32_t)(c + 16), r1);
                    tmem_ld_wait16(r0);
                    tmem_ld_wait16(r1);
                    const int n = q0 + c;
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[j] = __uint_as_float(r0[j]);
                        v[16 + j] = __uint_as_float(r1[j]);
                    }
                    if (bias && n < N) bias_add32(v, lbs[c / 32]);  // warp-uniform condition
                    if (m < M && n < N) {
                        uint16_t *o = out + (size_t)m * N + n;
                        if (vec_ok && n + 32 <= N) {
#pragma unroll
                            for (int j = 0; j < 32; j += 8) OutStore<uint16_t>::eight(o + j, v + j);
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (n + j < N) OutStore<uint16_t>::one(o + j, v[j]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[b]);
            if (!have) break;
        }
    } else {
        // ---- scale staging: warps 6..9, one per TMEM lane quarter ----
        const int quarter = warp & 3;
        const uint32_t qlane = (uint32_t)(quarter * 32) << 16;
        constexpr int PD = 2;  // chunks whose words are in flight
        int it = 0;
        bool stop = false;
        for (int t = blockIdx.x; t < num_tiles && !stop; t += gridDim.x) {
            int p0, q0;
            fp4_coords(t, p_tiles, q_tiles, group, BQ, p0, q0);
            const int ra = p0 + quarter * 32 + lane;  // this lane's x row (A scales, its own quarter)
            const uint8_t *pa = xs + (size_t)(ra < M ? ra : 0) * nb;
            const uint8_t *pb = ws + (size_t)(q0 + lane) * nb;  // W rows 32j + lane (every quarter holds them)
            uint2 a[PD], b[PD][kBcols];
#pragma unroll
            for (int d = 0; d < PD; ++d) {
                a[d] = scale_words<W>(pa, d, nb, ra < M);
#pragma unroll
                for (int j = 0; j < kBcols; ++j)
                    b[d][j] = scale_words<W>(pb + (size_t)(32 * j) * nb, d, nb, q0 + 32 * j + lane < N);
            }
            for (int c = 0; c < C; ++c, ++it) {
                const int s = it % stages;
                if (it >= stages && !mbar_wait(&sh.empty[s], ((it / stages) - 1) & 1, status, kSiteScale)) {
                    atomicExch(&sh.aborted, 1);
                    stop = true;
                }
                stop = __any_sync(0xffffffffu, stop) || *((volatile int32_t *)&sh.aborted);
                if (__any_sync(0xffffffffu, stop)) {
                    stop = true;
                    break;
                }
                const uint32_t sf = tmem + (uint32_t)(kSf + kSlot * s) + qlane;
                tmem_st4(sf, a[0].x, a[0].x, a[0].x, a[0].x);  // column `quarter` of the four is the one read
                tmem_st4(sf + 8, a[0].y, a[0].y, a[0].y, a[0].y);
#pragma unroll
                for (int j = 0; j < kBcols; j += 4) {
                    tmem_st4(sf + 16 + j, b[0][j].x, b[0][j + 1].x, b[0][j + 2].x, b[0][j + 3].x);
                    tmem_st4(sf + 24 + j, b[0][j].y, b[0][j + 1].y, b[0][j + 2].y, b[0][j + 3].y);
                }
#pragma unroll
                for (int d = 0; d + 1 < PD; ++d) {
                    a[d] = a[d + 1];
#pragma unroll
                    for (int j = 0; j < kBcols; ++j) b[d][j] = b[d + 1][j];
                }
                a[PD - 1] = scale_words<W>(pa, c + PD, nb, ra < M);
#pragma unroll
                for (int j = 0; j < kBcols; ++j)
                    b[PD - 1][j] = scale_words<W>(pb + (size_t)(32 * j) * nb, c + PD, nb, q0 + 32 * j + lane < N);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.sfull[s]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        for (int i = sh.consumed; i < sh.issued; ++i)
            mbar_wait(&sh.full[i % stages], (i / stages) & 1, status, kSiteDrain);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

int fp4_smem_bytes(int stages, int bq) {
    const int need = 1024 + stages * stage_bytes(bq) + (int)sizeof(TileShared);
    return need > 116 * 1024 ? need : 116 * 1024;  // one CTA per SM (each allocates all 512 TMEM columns)
}

int fp4_max_stages(int bq) {
    const int fit = (232448 - 1024 - (int)sizeof(TileShared)) / stage_bytes(bq);
    return fit < kMaxStages ? fit : kMaxStages;
}

using TileFn = void (*)(const CUtensorMap, const CUtensorMap, const uint8_t *, const uint8_t *, const uint16_t *,
                        uint16_t *, int, int, int, int, int, int32_t *);

template <int BQ>
TileFn pick_tile(int w) {
    return w == 8 ? mxfp4_tile_kernel<BQ, 8> : w == 4 ? mxfp4_tile_kernel<BQ, 4> : mxfp4_tile_kernel<BQ, 1>;
}

}  // namespace

int init_mxfp4_tile() {
    for (int bq : {128, 256})
        for (int w : {8, 4, 1}) {
            const int e = (int)cudaFuncSetAttribute(bq == 128 ? pick_tile<128>(w) : pick_tile<256>(w),
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    fp4_smem_bytes(fp4_max_stages(bq), bq));
            if (e) return e;
        }
    return 0;
}

int launch_mxfp4_tile(const void *xq, const void *xs, const void *wq, const void *ws, const void *bias, void *out,
                      int M, int N, int K, int bq, int num_sms, uint32_t flags, void *stream, int32_t *status) {
    const int stages = fp4_max_stages(bq);
    CUtensorMap tx, tw;  // 128-byte rows of 256 codes
    int r = make_tmap_u8_2d(&tx, xq, (uint64_t)M, (uint64_t)(K / 2), kBP, kChunkBytes, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (r) return (int)cudaErrorInvalidValue;
    r = make_tmap_u8_2d(&tw, wq, (uint64_t)N, (uint64_t)(K / 2), (uint32_t)bq, kChunkBytes, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (r) return (int)cudaErrorInvalidValue;
    const long long tiles = (long long)((M + kBP - 1) / kBP) * ((N + bq - 1) / bq);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < num_sms ? tiles : num_sms));
    cfg.blockDim = dim3(kMxfp4TileThreads);
    cfg.dynamicSmemBytes = (size_t)fp4_smem_bytes(stages, bq);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uintptr_t a = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws) | (uintptr_t)(K / 32);
    const int w = a % 8 == 0 ? 8 : a % 4 == 0 ? 4 : 1;
    return (int)cudaLaunchKernelEx(&cfg, bq == 128 ? pick_tile<128>(w) : pick_tile<256>(w), tx, tw,
                                   static_cast<const uint8_t *>(xs), static_cast<const uint8_t *>(ws),
                                   static_cast<const uint16_t *>(bias), static_cast<uint16_t *>(out), M, N, K, stages, 8,
                                   status);
}

}  // namespace bf16l
