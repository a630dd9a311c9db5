// mxfp4_split.cu — the MXFP4 linear where reading W, or filling the SMs, sets the
// cost: from one token to a few hundred.
//
// W rows sit on the MMA's M side (tcgen05.mma.kind::mxf4.block_scale, 128 rows), NT
// (16 to 64) tokens on its N side, and K is cut into runs for the S CTAs of a
// cluster, so that a few thousand W rows still occupy every SM.  The weight goes from
// HBM to the tensor core without passing a register: widening 4-bit codes for
// mma.sync took 50 to 100 instructions for each 512 codes and left 1 x 14336 x 4096 at
// 17 us and 16 x 14336 x 4096 at 31 us.
//
//   * a ring stage is one 256-code chunk (128-byte swizzle rows, TMA): 16 KB of W and
//     NT * 128 bytes of x;
//   * warp 0: TMA producer; warp 1: MMA issuer (four a chunk, two 32-code scale blocks
//     each), TMEM; warps 2-5: scales, then the epilogue (TMEM lane quarter = warp % 4);
//     warps 6 and 7 help to stage x and to join the sums;
//   * scales: thread i reads eight bytes (a chunk) of W row i, and each warp those of
//     all NT tokens (every lane quarter needs them), kAhead chunks ahead, and writes
//     the words to one of the TMEM slots: W words at columns 0 and 8 of the slot,
//     token words at 16 and 24.  Rows that do not start on 8-byte boundaries (K % 256) go
//     by cp.async in 16-byte blocks, each row's once for the CTA, and are shifted on the
//     way out of shared memory: from codes 558 x 2112 x 6176 16.8 us, 13 x 5760 x 2880 6.7
//     (33.6 and 7.2 by words from the row's first byte on: three loads for a chunk and row,
//     each a cache line per lane);
//   * M <= 16: all threads put the CTA's whole run of x into shared memory, in the layout
//     that TMA would have written, while the first W chunks are on their way: from codes
//     (a TMA box that is mostly past M is slow: 1 x 14336 x 4096 16 us with it), or
//     quantising a bf16 x: no kernel and no memory before this one, and the same bits;
//   * the CTAs of a cluster leave their fp32 sums [token][row] in shared memory, and
//     after a cluster barrier each adds the S sums of its share of the tokens, in rank
//     order, adds the bias and rounds: the order never changes;
//   * K past its end: codes are zero (TMA fill), scale bytes 1.0.
//
// This form is bound by its latencies in series: launch, TMEM and barriers 2.0 us, cold
// codes 1 to 1.5, scales 1.2, the join 0.5 (16 tokens) to 2 (64).  From codes / from bf16,
// weights not in L2: 1 x 2112 x 7168 6.0 / 6.2 us, 16 x 2112 x 7168 6.8 / 8.3, 1 x 14336 x
// 4096 10.0 / 9.8 (3.2 TB/s), 64 x 14336 x 4096 11.4 / 13.4.  They are not the product's
// own bound: the bf16 linear, on nearly four times the bytes, takes 5.3, 7.4, 18.3 and 24.0.
// Measured and not taken: W's rows asked into L2 before the wait for the previous kernel (0
// to 1 us slower), TMA boxes issued by a lane per stage (no change), scale words asked for
// before x is staged (-0.4 to +0.3 us), 128-token tiles (128 x 2112 x 7168 9.9 us, 8.4 with
// 64).
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

constexpr int kRowsW = 128, kChunkBytes = 128, kChunkBlocks = 8;
constexpr int kWBytes = kRowsW * kChunkBytes;
constexpr int kThreads = 256;
constexpr int kMaxSplit = 8, kMaxStages = 8;
constexpr int kSlotCols = 32;
constexpr int kAhead = 4;
constexpr int kRaw = 4;  // blocks of a shifted scale row in shared memory

// ... and their bytes: of 128 W rows, and of the tokens where no staging has brought them.
__host__ __device__ constexpr int raw_rows(int nt) { return nt == 16 ? kRowsW : kRowsW + nt; }
__host__ __device__ constexpr int raw_bytes(int nt) { return kRaw * 16 * raw_rows(nt); }

template <int NT>
struct Split {
    static constexpr int kSlots = NT <= 32 ? 3 : 2;
    static constexpr int kCols = 128;  // TMEM columns
    static constexpr int kSfCol = kCols - kSlots * kSlotCols;
    static constexpr int kXBytes = NT * kChunkBytes;
    static_assert(kSfCol >= NT, "TMEM columns");
};

// The ring, which later holds the sums of NT tokens.
__host__ __device__ constexpr int ring_bytes(int nt, int stages, int stage) {
    return stages * stage > nt * kRowsW * 4 ? stages * stage : nt * kRowsW * 4;
}

struct SplitArgs {
    const void *x;         // bf16, or codes
    const uint8_t *xs, *ws;
    const uint16_t *bias;
    uint16_t *out;
    int M, N, K, S, m_tiles, stages;
    int32_t *status;
    int w_early;
};

struct SplitShared {
    uint64_t full[kMaxStages], empty[kMaxStages], sfull[kMaxStages], acc_full;
    uint32_t tmem_base;
    int32_t aborted, issued, consumed;
};

// NT: tokens of a tile.  BF16: x is bf16 and is quantised here (NT == 16).  SHIFTED: scale rows do not all start on
// 8-byte boundaries (K % 256, or the tensors' start).  The way through shared memory would do for the others too, and
// gains with many chunks to a CTA (300 x 2112 x 6144 11.6 us, 12.4 by 8-byte loads), but costs where calls are short
// (64 x 2112 x 7168 8.0 and 7.7, 64 x 14336 x 4096 12.7 and 11.4).
template <int NT, bool BF16, bool SHIFTED>
__global__ void __launch_bounds__(kThreads, 2)
    mxfp4_split_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                       const SplitArgs a) {
    using T = Split<NT>;
    constexpr bool kStaged = NT == 16;  // x by the threads rather than by TMA
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nb = a.K >> 5, C = (nb + kChunkBlocks - 1) / kChunkBlocks;
    const int rank = a.S > 1 ? (int)cluster_ctarank() : 0;
    const int tile = (int)blockIdx.x / a.S;  // token tiles of one W tile follow each other
    const int n0 = (tile / a.m_tiles) * kRowsW, m0 = (tile % a.m_tiles) * NT;
    const int c0 = mul_div(C, rank, a.S), nc = mul_div(C, rank + 1, a.S) - c0;  // this CTA's chunks
    const int tokens = a.M - m0 < NT ? a.M - m0 : NT;
    // stages of W (and of x where TMA brings it); then, where x is staged, its whole run and the scale bytes
    constexpr int kStage = kWBytes + (kStaged ? 0 : T::kXBytes);
    const int stages = a.stages;
    uint8_t *xrun = base + ring_bytes(NT, stages, kStage);  // [nc][NT][128], swizzled
    const int nc_most = (C + a.S - 1) / a.S;
    uint8_t *xscale = xrun + nc_most * T::kXBytes;          // [nc][NT][8]
    uint8_t *after = kStaged ? xscale + nc_most * NT * 8 : xrun;
    uint4(*raw_scales)[raw_rows(NT)] = reinterpret_cast<uint4(*)[raw_rows(NT)]>(after);  // SHIFTED: [kRaw][row]
    SplitShared &sh = *reinterpret_cast<SplitShared *>(after + (SHIFTED ? raw_bytes(NT) : 0));

    if (tid == 0) {
        tma_prefetch_desc(&tm_w);
        if (!kStaged) tma_prefetch_desc(&tm_x);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int s = 0; s < T::kSlots; ++s) mbar_init(&sh.sfull[s], 4);  // one arrival per scale warp
        mbar_init(&sh.acc_full, 1);
        sh.aborted = 0;
        sh.issued = 0;
        sh.consumed = 0;
        fence_barrier_init();
    }
    // the codes of chunk i into its stage
    auto load = [&](int i) {
        const int s = i % stages;
        uint8_t *st = base + s * kStage;
        mbar_arrive_expect_tx(&sh.full[s], kStage);
        tma_load_2d(st, &tm_w, &sh.full[s], (c0 + i) * kChunkBytes, n0);
        if (!kStaged) tma_load_2d(st + kWBytes, &tm_x, &sh.full[s], (c0 + i) * kChunkBytes, m0);
    };
    int first = 0;  // chunks that the producer has already asked for
    if (!kStaged || !a.w_early) pdl_wait();
    if (tid == 0)
        for (; first < stages && first < nc; ++first) load(first);
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, T::kCols);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();  // x may be written, and out still read, by the previous kernel
    if (kStaged && BF16) {
        // item: eight codes (a quad holds a block); the loads of kBatch items of a thread go out together
        constexpr int kBatch = 8;
        // (the tokens of the tile past M stay as they are: their columns of the accumulator are not read)
        const int per = nc * kChunkBlocks * 4, items = tokens * per;  // multiples of 32: warps stay together
        for (int i0 = tid; i0 < items; i0 += kBatch * kThreads) {
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kThreads, tok = i / per, r = i - tok * per, b = c0 * kChunkBlocks + (r >> 2);
                v[k] = (i < items && b < nb)
                           ? __ldg(static_cast<const uint4 *>(a.x) + ((size_t)(m0 + tok) * nb + b) * 4 + (r & 3))
                           : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * kThreads, tok = i / per, r = i - tok * per;
                if (i >= items) break;
                uint32_t s;
                const uint32_t w = mxfp4_quant_vec(v[k], 0xFu << (lane & 28), s);
                const int c = r >> 5, u = (r >> 2) & 7;  // chunk, 16-byte unit of its row (a block)
                uint8_t *to = xrun + c * T::kXBytes + tok * 128 + 16 * (u ^ (tok & 7)) + 4 * (r & 3);
                *reinterpret_cast<uint32_t *>(to) = w;
                if ((r & 3) == 0) xscale[(c * NT + tok) * 8 + u] = (uint8_t)s;
            }
        }
    } else if (kStaged) {
        const int per = nc * kChunkBlocks;  // item: a block, 16 bytes of codes and a scale byte
        for (int i = tid; i < tokens * per; i += kThreads) {
            const int tok = i / per, r = i - tok * per, b = c0 * kChunkBlocks + r, c = r >> 3, u = r & 7;
            const bool in = b < nb;
            const size_t at = (size_t)(m0 + tok) * nb + b;
            *reinterpret_cast<uint4 *>(xrun + c * T::kXBytes + tok * 128 + 16 * (u ^ (tok & 7))) =
                in ? __ldg(static_cast<const uint4 *>(a.x) + at) : make_uint4(0u, 0u, 0u, 0u);
            xscale[(c * NT + tok) * 8 + u] = in ? __ldg(a.xs + at) : (uint8_t)127;
        }
    }
    if (kStaged) fence_proxy_async_smem();  // the MMAs read xrun through the async proxy
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;

    if (warp == 0) {
        if (lane == 0) {  // ---- TMA producer ----
            int i = first;
            for (; i < nc; ++i) {
                if (i >= stages && !mbar_wait(&sh.empty[i % stages], ((i / stages) - 1) & 1, a.status, kSiteEmpty)) {
                    atomicExch(&sh.aborted, 1);
                    break;
                }
                if (*((volatile int32_t *)&sh.aborted)) break;
                load(i);
            }
            sh.issued = i;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {  // ---- MMA issuer ----
            int i = 0;
            for (; i < nc; ++i) {
                const int s = i % stages, f = i % T::kSlots;
                if (!mbar_wait(&sh.full[s], (i / stages) & 1, a.status, kSiteFull) ||
                    !mbar_wait(&sh.sfull[f], (i / T::kSlots) & 1, a.status, kSiteScale)) {
                    atomicExch(&sh.aborted, 1);
                    break;
                }
                tc_fence_after();
                uint8_t *st = base + s * kStage;
                const uint64_t wdesc = smem_desc_sw128(smem_u32(st));
                const uint64_t xdesc = smem_desc_sw128(smem_u32(kStaged ? xrun + i * T::kXBytes : st + kWBytes));
                const uint32_t sf = tmem + (uint32_t)(T::kSfCol + kSlotCols * f);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)  // 64 codes, two scale blocks
                    mma_mxf4(tmem, wdesc + 2 * kk, xdesc + 2 * kk, idesc_mxf4_f32(kRowsW, NT, 2 * (kk & 1)),
                             sf + 8 * (kk >> 1), sf + 16 + 8 * (kk >> 1), (i > 0 || kk > 0) ? 1u : 0u);
                mma_commit(&sh.empty[s]);
            }
            sh.consumed = i;
            if (i < nc)
                mbar_arrive(&sh.acc_full);
            else
                mma_commit(&sh.acc_full);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ---- scales ----
        const int quarter = warp & 3;
        const uint32_t slot0 = tmem + (uint32_t)T::kSfCol + ((uint32_t)(quarter * 32) << 16);
        constexpr int kTw = (NT + 31) / 32;  // token words per lane
        const int row = n0 + 32 * quarter + lane;
        const uint2 one = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        // the slot of chunk i is free when the MMAs of the chunk kSlots before are done
        auto slot_free = [&](int i) {
            const int old = i - T::kSlots;
            const bool ok =
                old < 0 || mbar_wait(&sh.empty[old % stages], (old / stages) & 1, a.status, kSiteScale);
            if (!__any_sync(0xFFFFFFFFu, !ok || *((volatile int32_t *)&sh.aborted))) return true;
            atomicExch(&sh.aborted, 1);
            return false;
        };
        auto put = [&](int i, const uint2 &w, const uint2 (&x)[kTw]) {
            const uint32_t sf = slot0 + (uint32_t)(kSlotCols * (i % T::kSlots));
            tmem_st4(sf, w.x, w.x, w.x, w.x);  // column `quarter` of the four is the one read
            tmem_st4(sf + 8, w.y, w.y, w.y, w.y);
            constexpr int l = kTw - 1;
            tmem_st4(sf + 16, x[0].x, x[l < 1 ? l : 1].x, x[l < 2 ? l : 2].x, x[l].x);
            tmem_st4(sf + 24, x[0].y, x[l < 1 ? l : 1].y, x[l < 2 ? l : 2].y, x[l].y);
        };
        auto arrive = [&](int i) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.sfull[i % T::kSlots]);
        };
        auto staged_words = [&](int i) {  // of token `lane`, chunk i of the run
            return lane < NT && i < nc ? *reinterpret_cast<const uint2 *>(xscale + (i * NT + lane) * 8) : one;
        };
        if constexpr (SHIFTED) {
            // The rows' bytes from this run's first on, in 16-byte blocks counted from the boundary before: thread t
            // asks for those of W row t and of token t, three blocks ahead.
            const int t = tid - 64, most = min(nb - kChunkBlocks * c0, kChunkBlocks * nc);
            const uint8_t *whi = a.ws + (size_t)a.N * nb, *xhi = a.xs + (size_t)a.M * nb;
            const uint8_t *pw = a.ws + (size_t)(n0 + t) * nb + kChunkBlocks * c0;  // (read where the row exists)
            const uint8_t *px = a.xs + (size_t)(m0 + t) * nb + kChunkBlocks * c0;
            auto off = [](const uint8_t *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15u); };
            // how many blocks the rows have (none where there is no such row)
            const int kw = n0 + t < a.N ? (off(pw) + most + 15) / 16 : 0;
            const int kx = !kStaged && t < tokens ? (off(px) + most + 15) / 16 : 0;
            auto ask = [&](int k) {
                uint4 *to = raw_scales[k % kRaw];
                if (k < kw) copy_block(&to[t], pw - off(pw) + 16 * k, a.ws, whi);
                if (k < kx) copy_block(&to[kRowsW + t], px - off(px) + 16 * k, a.xs, xhi);
                cp_async_commit();
            };
            // what this lane takes of them: W row 32 quarter + lane, tokens 32 j + lane
            constexpr int kTake = kStaged ? 1 : 1 + kTw;
            int at[kTake], m[kTake], n[kTake];
#pragma unroll
            for (int r = 0; r < kTake; ++r) {
                const int i = r == 0 ? 32 * quarter + lane : 32 * (r - 1) + lane;
                at[r] = r == 0 ? i : kRowsW + i;
                m[r] = off((r == 0 ? a.ws + (size_t)(n0 + i) * nb : a.xs + (size_t)(m0 + i) * nb) + kChunkBlocks * c0);
                n[r] = (r == 0 ? n0 + i < a.N : i < tokens) ? most : 0;
            }
            for (int k = 0; k < kRaw - 1; ++k) ask(k);
            // A warp that gave up goes on through the barriers, so that no other one waits for it there.
            bool stop = false;
            for (int i0 = 0; i0 < nc; i0 += 2) {
                const int k = i0 / 2;
                cp_async_wait<kRaw - 3>();  // this thread's block k + 1 and those before it are there,
                named_barrier(1, 4 * 32);   // and the others' too; block k - 1 has been read
                ask(k + kRaw - 1);
                if (stop) continue;
                uint4 q[kTake];
#pragma unroll
                for (int r = 0; r < kTake; ++r)
                    q[r] = scales_until(
                        shift_blocks(raw_scales[k % kRaw][at[r]], raw_scales[(k + 1) % kRaw][at[r]], m[r]),
                        n[r] - 16 * k);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (i0 + h >= nc || stop) break;
                    if (!slot_free(i0 + h)) {
                        stop = true;
                        break;
                    }
                    uint2 x[kTw];
#pragma unroll
                    for (int j = 0; j < kTw; ++j) {
                        const uint4 &v = q[kStaged ? 0 : 1 + j];
                        x[j] = kStaged ? staged_words(i0 + h) : h ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y);
                    }
                    put(i0 + h, h ? make_uint2(q[0].z, q[0].w) : make_uint2(q[0].x, q[0].y), x);
                    arrive(i0 + h);
                }
            }
            cp_async_wait<0>();
        } else {
            const uint8_t *wr = a.ws + (size_t)(row < a.N ? row : 0) * nb;
            const uint8_t *xr = kStaged ? nullptr : a.xs + (size_t)m0 * nb;
            auto w_words = [&](int i) {  // of this lane's W row, chunk i of the run
                return row < a.N && i < nc ? __ldg(reinterpret_cast<const uint2 *>(wr) + c0 + i) : one;
            };
            auto token_words = [&](int j, int i) {  // of token 32 j + lane, chunk i of the run
                if (kStaged) return staged_words(i);
                const int tok = 32 * j + lane;
                if (tok >= tokens || i >= nc) return one;
                return __ldg(reinterpret_cast<const uint2 *>(xr + (size_t)tok * nb) + c0 + i);
            };
            uint2 vw[kAhead], vx[kAhead][kTw];
#pragma unroll
            for (int d = 0; d < kAhead; ++d) {
                vw[d] = w_words(d);
#pragma unroll
                for (int j = 0; j < kTw; ++j) vx[d][j] = token_words(j, d);
            }
            bool stop = false;
            for (int i0 = 0; i0 < nc && !stop; i0 += kAhead) {
#pragma unroll
                for (int d = 0; d < kAhead; ++d) {
                    const int i = i0 + d;
                    if (i >= nc) break;
                    if (!slot_free(i)) {
                        stop = true;
                        break;
                    }
                    put(i, vw[d], vx[d]);
                    vw[d] = w_words(i + kAhead);
#pragma unroll
                    for (int j = 0; j < kTw; ++j) vx[d][j] = token_words(j, i + kAhead);
                    arrive(i);
                }
            }
        }
        // ---- epilogue: lane = W row, columns = tokens ----
        const bool ok = mbar_wait(&sh.acc_full, 0, a.status, kSiteAccum);
        tc_fence_after();
        const bool have = __all_sync(0xFFFFFFFFu, ok && !*((volatile int32_t *)&sh.aborted));
        if (have) {
            // [token][128 rows], over the ring: every chunk has been read
            float *sums = reinterpret_cast<float *>(base);
            const float bias = a.bias && row < a.N ? bf16_to_f32(__ldg(a.bias + row)) : 0.0f;
            const uint32_t acc = tmem + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                if (c >= tokens) break;
                uint32_t r[16];
                tmem_ld16(acc + (uint32_t)c, r);
                tmem_ld_wait16(r);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float v = __uint_as_float(r[j]);
                    if (a.S > 1)
                        sums[(c + j) * kRowsW + 32 * quarter + lane] = v;
                    else if (c + j < tokens && row < a.N)
                        a.out[(size_t)(m0 + c + j) * a.N + row] = f32_to_bf16(v + bias);
                }
            }
        }
        tc_fence_before();
    }
    if (a.S > 1) {
        cluster_sync();  // every CTA's sums are in its shared memory
        const bool have = *((volatile int32_t *)&sh.aborted) == 0;
        const int row = n0 + 4 * lane;  // a warp takes a token at a time, a lane four rows of it
        const bool vec = a.N % 4 == 0;
        float bias[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (a.bias && row + j < a.N) bias[j] = bf16_to_f32(__ldg(a.bias + row + j));
        for (int tok = rank + a.S * warp; have && tok < tokens; tok += a.S * (kThreads / 32)) {
            const uint32_t at = smem_u32(base) + (uint32_t)(tok * kRowsW + 4 * lane) * 4u;
            float4 v[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                if (r < a.S) v[r] = ld_dsmem_f4(mapa_shared(at, (uint32_t)r));
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                if (r < a.S) s[0] += v[r].x, s[1] += v[r].y, s[2] += v[r].z, s[3] += v[r].w;  // ranks in order
            uint16_t *o = a.out + (size_t)(m0 + tok) * a.N + row;
            if (vec && row + 3 < a.N) {
                OutStore<uint16_t>::four(o, s[0] + bias[0], s[1] + bias[1], s[2] + bias[2], s[3] + bias[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (row + j < a.N) o[j] = f32_to_bf16(s[j] + bias[j]);
            }
        }
        cluster_sync();  // nobody exits while its sums are still read
    } else {
        __syncthreads();
    }
    if (tid == 0) {  // copies that were issued but never consumed (only after a timeout)
        for (int i = sh.consumed; i < sh.issued; ++i)
            if (!mbar_wait(&sh.full[i % stages], (i / stages) & 1, a.status, kSiteDrain)) break;
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, T::kCols);
    }
}

int ceil_div(int a, int b) { return a / b + (a % b != 0); }  // (a + b - 1 may not fit)

using SplitFn = void (*)(const CUtensorMap, const CUtensorMap, const SplitArgs);

template <bool SHIFTED>
SplitFn pick_by(int nt, bool bf16) {
    if (nt == 16) return bf16 ? mxfp4_split_kernel<16, true, SHIFTED> : mxfp4_split_kernel<16, false, SHIFTED>;
    return nt == 32 ? mxfp4_split_kernel<32, false, SHIFTED> : mxfp4_split_kernel<64, false, SHIFTED>;
}

SplitFn pick_split(int nt, bool bf16, bool shifted) {
    return shifted ? pick_by<true>(nt, bf16) : pick_by<false>(nt, bf16);
}

constexpr int kMaxSmem = 227 * 1024;
// Two CTAs to an SM, or one, and none beside a kernel that takes all of TMEM (those ask for 116 KB or more): the
// CTAs of a cluster wait for one another, so none of them may wait for TMEM that another cluster's CTA holds.
constexpr int kHalfSmem = 112 * 1024, kHalfSmemMost = 113 * 1024;

long long split_smem(int nt, int stages, int S, int K, bool shifted) {
    const int nc = ceil_div(ceil_div(K, 256), S);
    long long n = 1024 + ring_bytes(nt, stages, kWBytes + (nt == 16 ? 0 : nt * kChunkBytes)) + (int)sizeof(SplitShared);
    if (nt == 16) n += (long long)nc * nt * (kChunkBytes + 8);  // (a run of x: past 32 bits where K is two billion)
    if (shifted) n += raw_bytes(nt);
    return n > kHalfSmem ? n : kHalfSmem;
}

int split_slots(int nt) { return nt <= 32 ? Split<32>::kSlots : Split<64>::kSlots; }

Mxfp4SplitPlan plan_for(int tokens, int M, int N, int K, int num_sms, bool shifted) {
    Mxfp4SplitPlan p;
    const int C = ceil_div(K, 256), n_tiles = ceil_div(N, kRowsW);
    p.tokens = tokens;
    p.m_tiles = ceil_div(M, p.tokens);
    // K over S CTAs: microseconds from timings of 40 shapes (1 to 512 tokens, 256 to 14336 rows).  A chunk takes
    // about 0.4 where every SM has at most one CTA, and as much longer as there are more; joining S sums costs more
    // with S, and with the tokens where S is 8.  64 x 2112 x 7168: S = 1, 2, 4, 8 take 16.0, 10.7, 7.7, 8.6 us; 16 x
    // 2112 x 7168: 16.7, 10.8, 8.0, 7.0; 1 x 14336 x 4096: 11.7, 9.9, 13.0, 19.0.
    const float tiles = (float)n_tiles * (float)p.m_tiles;
    float best = 0.0f;
    for (int S = 1; S <= kMaxSplit && S <= C; S *= 2) {
        const float load = tiles * (float)S / (float)num_sms;
        const float join = S == 1 ? 0.0f : S == 2 ? 0.3f : S == 4 ? 0.7f : 0.7f + 0.03f * (float)p.tokens;
        const float t = 0.4f * (float)ceil_div(C, S) * (load > 1.0f ? load : 1.0f) + join;
        // (to compare with the pair form: just above one CTA to an SM the slowest SM has two; 558 x 2112 x 6144, 153
        // tiles: 15.5 us here, 12.8 in pairs)
        if (S == 1 || t < best) best = t, p.split = S, p.estimate = load > 1.0f && load < 1.4f ? t * 1.4f / load : t;
    }
    const int nc = ceil_div(C, p.split), slots = split_slots(p.tokens);
    const int most = tiles * (float)p.split > (float)num_sms ? kHalfSmemMost : kMaxSmem;
    p.stages = nc < kMaxStages ? nc : kMaxStages;
    // (with fewer stages than scale slots a slot's wait could miss a turn of the stage's barrier)
    while (p.stages > slots && split_smem(p.tokens, p.stages, p.split, K, shifted) > most) --p.stages;
    p.smem = split_smem(p.tokens, p.stages, p.split, K, shifted);
    return p;
}

}  // namespace

Mxfp4SplitPlan mxfp4_split_plan(int M, int N, int K, int num_sms, bool shifted) {
    // One plan whatever the device's SMs: codes, a bf16 x and the workspace's size are asked for apart, and the first two
    // have to sum in one order.
    if (M <= 16) num_sms = kGb300Sms;
    // Where a run of x does not fit (K of 200000 and more): by TMA, stage by stage, whatever the scales' alignment.
    if (M <= 16 && plan_for(16, M, N, K, num_sms, true).smem <= kMaxSmem)
        return plan_for(16, M, N, K, num_sms, shifted);
    return plan_for(M <= 32 ? 32 : 64, M, N, K, num_sms, shifted);
}

bool mxfp4_split_quantises(int M, int N, int K) { return mxfp4_split_plan(M, N, K, kGb300Sms, true).tokens == 16; }

int init_mxfp4_split() {
    for (bool shifted : {false, true})
        for (int nt : {16, 32, 64})
            for (bool b : {false, true}) {
                if (b && nt > 16) continue;
                const int e = (int)cudaFuncSetAttribute(pick_split(nt, b, shifted),
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
                if (e) return e;
            }
    return 0;
}

int launch_mxfp4_split(const void *x, const void *xs, const void *wq, const void *ws, const void *bias, void *out,
                       int M, int N, int K, int num_sms, uint32_t flags, void *stream, int32_t *status) {
    const bool bf16 = xs == nullptr;
    const uintptr_t al =
        (bf16 ? 0 : reinterpret_cast<uintptr_t>(xs)) | reinterpret_cast<uintptr_t>(ws) | (uintptr_t)(K / 32);
    const bool shifted = al % 8 != 0;
    const Mxfp4SplitPlan p = mxfp4_split_plan(M, N, K, num_sms, shifted);
    CUtensorMap tx = {}, tw;  // 128-byte rows of 256 codes
    int r = make_tmap_u8_2d(&tw, wq, (uint64_t)N, (uint64_t)(K / 2), kRowsW, kChunkBytes, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (r) return (int)cudaErrorInvalidValue;
    if (p.tokens > 16) {
        r = make_tmap_u8_2d(&tx, x, (uint64_t)M, (uint64_t)(K / 2), (uint32_t)p.tokens, kChunkBytes,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
        if (r) return (int)cudaErrorInvalidValue;
    }
    SplitArgs a = {x,
                   static_cast<const uint8_t *>(xs),
                   static_cast<const uint8_t *>(ws),
                   static_cast<const uint16_t *>(bias),
                   static_cast<uint16_t *>(out),
                   M,
                   N,
                   K,
                   p.split,
                   p.m_tiles,
                   p.stages,
                   status,
                   w_early_of(flags)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ceil_div(N, kRowsW) * p.m_tiles * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)p.smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return (int)cudaLaunchKernelEx(&cfg, pick_split(p.tokens, bf16, shifted), tx, tw, a);
}

}  // namespace bf16l
