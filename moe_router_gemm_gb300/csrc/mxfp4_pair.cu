// mxfp4_pair.cu — the MXFP4 linear as a dense contraction: CTA pairs
// (tcgen05.mma.cta_group::2.kind::mxf4.block_scale) on 256 x 256 tiles.
//
//   * cluster of 2; a ring stage is one 256-code chunk (128-byte swizzle rows, TMA)
//     of this CTA's own 128 x rows and 128 W rows, 32 KB; the even CTA (the leader)
//     issues every MMA: four per stage, two 32-code scale blocks each;
//   * warp 0: TMA producer; warp 1: MMA issuer (leader), TMEM; warps 2-9: epilogue;
//     warps 10-13: scales.  A stage is full when both CTAs' 64 KB have landed and the
//     eight scale warps have arrived on the leader's barrier;
//   * scales: thread i of the scale warps reads 16 scale bytes (two chunks) of x row
//     i and of W rows i and i + 128 of the tile, two steps ahead.  The W bytes go
//     through shared memory, since every TMEM lane quarter needs all 256 rows'; each
//     warp writes its quarter of a step's two slots with tcgen05.st (one wait and one
//     arrival for both: 8192 x 7168 x 7168 135.3 us a chunk at a time, 133 so).  Reading
//     each row once per CTA, 16 bytes at a time, matters: a row's bytes are a cache line
//     of their own.  Rows that do not start on 16-byte boundaries (K % 512) go by
//     cp.async, whole blocks, and are shifted on the way out of shared memory: 8192 x
//     7168 x 2880 81 us, x 6176 158 (117 and 259 by words from the row's first byte on;
//     blocks in registers 87 and 170, which are too few to keep loads in flight);
//   * TMEM: accumulators at columns 0 and 128, 256 columns each, taken in turn: they
//     share columns 128-255, which the epilogue empties first, so the next tile's
//     MMAs start when half of this one is out; four scale slots of 32 columns (x words
//     at 0 and 8, W words at 16 and 24: every address a multiple of 8) from 384;
//   * epilogue, N % 8 == 0: 32 x 32 pieces through shared memory and TMA stores (each
//     lane storing its own row's 16-byte pieces takes a line per lane and held
//     8192 x 7168 x 7168 at 174 us).  Other N, whose rows start on no 16-byte boundary:
//     rows of 64 columns through shared memory, a warp's store taking whole rows.
//     6152 x N x 32: N = 12064 42 us; 12060 (8-byte stores) 53, 12062 (4-byte) 56, 12061
//     70, where a lane storing its own row took 680.  Rows shifted in shared memory to
//     their place in out's 16-byte lines, 16-byte stores and the rest by elements: 84, 85
//     and 89: the shifts and single elements cost more instructions than they save;
//   * K past its end: codes are zero (TMA fill), scale bytes 1.0.
//
// Measured and not taken (8192 x 7168 x 7168): arrivals released at cluster scope (they
// wait for the scale loads in flight) 384 us; scales copied by tcgen05.cp from shared
// memory, in order before their MMAs 196 us, a chunk ahead or between the MMAs 207 us
// (the copies hold up the MMAs behind them); two or three scale slots, which leave the
// accumulators fewer shared columns, 185 and 177 us against 174.
//
// Cross-CTA lifetime: a cluster barrier after set-up (every barrier exists before any
// remote arrival) and one before TMEM is freed and the CTAs exit.  Every wait is bounded.
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

constexpr int kHalf = 128;                  // rows of each operand per CTA and chunk
constexpr int kTileRows = 256;              // x rows, and W rows, of a pair tile
constexpr int kChunkBytes = 128;            // code bytes of a row per chunk (256 codes)
constexpr int kHalfBytes = kHalf * kChunkBytes;
constexpr int kStageBytes = 2 * kHalfBytes;
constexpr int kStages = 6;  // (five where scale rows are shifted: the memory of their blocks)
constexpr int kRaw = 4;     // blocks of a shifted scale row in shared memory
// W tiles of a raster group: 8192 x 7168 x 7168 takes 135.6 us with 4, 136.7 with 2, 138 with 8
constexpr int kGroup = 4;
constexpr int kSlots = 4, kSlotCols = 32;
constexpr int kSfCol = 512 - kSlots * kSlotCols;  // the scale slots' first column
constexpr int kAcc1Col = kSfCol - kTileRows;      // the second accumulator's first column
constexpr int kShared = kTileRows - kAcc1Col;     // columns that the accumulators share
static_assert(kShared == 128, "the epilogue empties 128 columns first");
constexpr int kEpiWarps = 8, kScaleWarps = 4;
constexpr int kPitch = 144;  // bytes of a shifted row of 64 columns: nine units; eight neighbouring rows' never collide
constexpr int kPieceBytes = 2560;
constexpr int kThreads = 32 * (2 + kEpiWarps + kScaleWarps);

// K % 32 == 0 (K + 255 may not fit an int).
__host__ __device__ constexpr int chunks_of(int K) { return K / 256 + (K % 256 != 0); }
static_assert(2 * kChunkBytes == 256, "two codes to a byte");
__host__ __device__ constexpr int tiles_of(int rows) { return rows / kTileRows + (rows % kTileRows != 0); }

template <bool SHIFTED>
struct PairShared {
    static constexpr int kStages = SHIFTED ? bf16l::kStages - 1 : bf16l::kStages;
    // an epilogue warp's 32 rows x 32 columns in bf16, 64-byte swizzle (first, so aligned), or 16 rows of kPitch bytes
    uint8_t piece[kEpiWarps][kPieceBytes];
    uint4 scales[2][kTileRows];
    uint4 raw[SHIFTED ? kRaw : 1][SHIFTED ? 3 : 1][kHalf];  // blocks of each scale thread's x row and two W rows
    uint64_t full[kStages];    // leader only: both CTAs' codes and scales of the stage are in shared memory
    uint64_t empty[kStages];   // both: the MMAs (and copies) reading the stage are done
    uint64_t acc_full[2];      // both: accumulator holds a finished tile
    uint64_t acc_shared;       // leader only: both CTAs' epilogues have the shared columns of a tile
    uint32_t tmem_base;
    int32_t bad_pair, aborted, issued, consumed;
};

__device__ __forceinline__ void pair_coords(int u, int p_tiles, int q_tiles, int &p0, int &q0) {
    const int per_group = kGroup * p_tiles;
    const int g = u / per_group, r = u - g * per_group;
    const int gq = (q_tiles - g * kGroup) < kGroup ? (q_tiles - g * kGroup) : kGroup;
    const int pi = r / gq, qi = g * kGroup + (r - pi * gq);
    p0 = pi * kTileRows;
    q0 = qi * kTileRows;
}

// 32 rows (one a lane) x 64 columns (p) to rows of out that start on no 16-byte boundary: sixteen rows at a time
// through shared memory, then T at a time, a store taking whole rows.  N, and so `cols` (64, or what is left of out),
// is a multiple of T's elements, or odd: then T is a word, every other row starts within one and goes to shared memory
// an element further on, and single elements at a row's ends are stored by themselves.
template <class T, bool ODD>
__device__ __forceinline__ void store_rows(uint16_t *o, uint8_t *piece, const uint32_t (&p)[32], int rows, int cols,
                                           int N, int lane) {
    constexpr int lanes = 128 / sizeof(T), at_once = 32 / lanes, each = sizeof(T) / 2;  // lanes: of a row
    const int s0 = ODD ? (int)(reinterpret_cast<uintptr_t>(o) >> 1) & 1 : 0;  // (row r: s0 ^ r & 1)
    const bool mine = ODD && ((s0 ^ lane) & 1);
#pragma unroll 1
    for (int r0 = 0; r0 < 32 && r0 < rows; r0 += 16, o += (size_t)16 * N) {
        __syncwarp();  // the rows before have been read
        if ((lane & 16) == r0) {
            uint32_t *q = reinterpret_cast<uint32_t *>(piece + kPitch * (lane & 15));
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                uint32_t t[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    t[j] = mine ? __funnelshift_l(k + j > 0 ? p[k + j - 1] : 0u, p[k + j], 16) : p[k + j];
                *reinterpret_cast<uint4 *>(q + k) = make_uint4(t[0], t[1], t[2], t[3]);
            }
            if (mine) q[32] = p[31] >> 16;
        }
        __syncwarp();
        const int have = min(rows - r0, 16);
        const int r1 = lane / lanes, u = lane % lanes;
        const uint8_t *from = piece + kPitch * r1 + (int)sizeof(T) * u;
        T v[16 / at_once];  // read before the first store, which they would have to wait for
#pragma unroll
        for (int i = 0; i < 16; i += at_once)
            v[i / at_once] = *reinterpret_cast<const T *>(from + kPitch * i + 4 * ((s0 ^ i) & ODD));
        // Odd N: what row lane / 2 has outside its words, its first element (even lanes) or its last (odd lanes).
        const int er = lane >> 1, es = (s0 ^ er) & 1;
        const int e = lane & 1 ? (es == (cols == 64) ? cols - 1 : -1) : es ? 0 : -1;
        uint16_t edge = 0;
        if (ODD && e >= 0) edge = *reinterpret_cast<const uint16_t *>(piece + kPitch * er + 2 * (e + es));
        uint16_t *to = o + (size_t)r1 * N + each * u;
#pragma unroll
        for (int i = 0; i < 16; i += at_once, to += (size_t)at_once * N) {
            const int sr = (s0 ^ i) & ODD;
            if (i + r1 < have && sr + each * u + each <= cols) *reinterpret_cast<T *>(to + sr) = v[i / at_once];
        }
        if (ODD && er < have && e >= 0) o[(size_t)er * N + e] = edge;
    }
}

// SHIFTED: scale rows do not all start on 16-byte boundaries (K % 512, or the tensors' start).  ALIGNED: rows of out do
// (N % 8 == 0); a kernel of its own, since the other rows' code costs it 2% (8192 x 7168 x 7168: 135.3 us, together
// 138.4).
template <bool SHIFTED, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1)
    mxfp4_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                      const __grid_constant__ CUtensorMap tm_out, const uint8_t *__restrict__ xs,
                      const uint8_t *__restrict__ ws, const uint16_t *__restrict__ bias, uint16_t *__restrict__ out,
                      int M, int N, int K, int32_t *status) {
    using Shared = PairShared<SHIFTED>;
    constexpr int kStages = Shared::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStageBytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int p_tiles = tiles_of(M), q_tiles = tiles_of(N);
    const int units = p_tiles * q_tiles;
    const int cl = (int)blockIdx.x >> 1, ncl = (int)gridDim.x >> 1;
    const int C = chunks_of(K);
    const int nb = K >> 5;

    if (tid == 0) {
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1 + 2 * kScaleWarps);  // the leader producer's arrive.expect_tx, the scale warps
            mbar_init(&sh.empty[s], 1);                   // the leader's multicast commit
        }
        mbar_init(&sh.acc_full[0], 1);
        mbar_init(&sh.acc_full[1], 1);
        mbar_init(&sh.acc_shared, 2 * kEpiWarps);
        sh.aborted = 0;
        sh.issued = 0;
        sh.consumed = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&sh.tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    // Both CTAs' barriers and TMEM exist before any cross-CTA arrival or copy.
    cluster_arrive_release();
    cluster_wait_acquire();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    // The pair MMA writes the same TMEM address in both CTAs: check that the joint
    // allocation gave both the same columns (each CTA reads the other's).
    if (tid == 0) {
        uint32_t other;
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(other)
                     : "r"(mapa_shared(smem_u32(&sh.tmem_base), rank ^ 1u))
                     : "memory");
        sh.bad_pair = other != tmem;
        if (other != tmem) record_timeout(status, kSitePairTmem);
    }
    __syncthreads();
    const bool bad_pair = sh.bad_pair != 0;  // the same verdict in both CTAs
    pdl_launch_dependents();
    pdl_wait();  // nothing is read before the previous kernel has finished

    if (bad_pair) {
        // nothing issued: fall through to the exit barrier
    } else if (warp == 0) {
        if (lane == 0) {  // ---- TMA producer (both CTAs) ----
            const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0);  // leader's full[0]
            int it = 0;
            for (int u = cl; u < units; u += ncl) {
                int p0, q0;
                pair_coords(u, p_tiles, q_tiles, p0, q0);
                const int ap = p0 + (int)rank * kHalf, bq = q0 + (int)rank * kHalf;
                for (int c = 0; c < C; ++c, ++it) {
                    const int s = it % kStages;
                    if (it >= kStages && !mbar_wait(&sh.empty[s], ((it / kStages) - 1) & 1, status, kSiteEmpty)) {
                        atomicExch(&sh.aborted, 1);
                        goto producer_done;
                    }
                    if (*((volatile int32_t *)&sh.aborted)) goto producer_done;
                    uint8_t *st = ring + s * kStageBytes;
                    if (leader) mbar_arrive_expect_tx(&sh.full[s], 2 * kStageBytes);
                    const uint32_t fb = full0 + (uint32_t)(s * sizeof(uint64_t));
                    tma_load_2d_pair(st, &tm_x, fb, c * kChunkBytes, ap);
                    tma_load_2d_pair(st + kHalfBytes, &tm_w, fb, c * kChunkBytes, bq);
                }
            }
        producer_done:
            sh.issued = it;
            // Every commit that arrives on this CTA's `empty` barriers has landed
            // before the exit barrier (the last kStages chunks).
            if (!*((volatile int32_t *)&sh.aborted)) {
                for (int i = (it > kStages ? it - kStages : 0); i < it; ++i)
                    if (!mbar_wait(&sh.empty[i % kStages], (i / kStages) & 1, status, kSiteDrain)) break;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {  // ---- MMA issuer (leader only) ----
            int it = 0, tile = 0;
            for (int u = cl; u < units; u += ncl, ++tile) {
                sh.consumed = it;
                const uint32_t acc = tmem + (uint32_t)((tile & 1) * kAcc1Col);
                // Both CTAs' epilogues have the columns that this accumulator shares with the previous tile's out,
                // and, as they take tiles in order, all of the tile before that.
                bool ok = tile == 0 || mbar_wait(&sh.acc_shared, (tile - 1) & 1, status, kSiteTmemEmpty);
                for (int c = 0; ok && c < C; ++c, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(&sh.full[s], (it / kStages) & 1, status, kSiteFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *st = ring + s * kStageBytes;
                    const uint64_t adesc = smem_desc_sw128(smem_u32(st));
                    const uint64_t bdesc = smem_desc_sw128(smem_u32(st + kHalfBytes));
                    const uint32_t sf = tmem + (uint32_t)(kSfCol + kSlotCols * (it % kSlots));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 64 codes, two scale blocks
                        mma_mxf4_pair(acc, adesc + 2 * kk, bdesc + 2 * kk,
                                      idesc_mxf4_f32(kTileRows, kTileRows, 2 * (kk & 1)), sf + 8 * (kk >> 1),
                                      sf + 16 + 8 * (kk >> 1), (c > 0 || kk > 0) ? 1u : 0u);
                    mma_commit_pair(&sh.empty[s], (uint16_t)0x3);
                }
                if (!ok) {  // release both epilogues at once
                    atomicExch(&sh.aborted, 1);
                    sh.consumed = it;
                    mbar_arrive(&sh.acc_full[tile & 1]);
                    mbar_arrive_cluster(mapa_shared(smem_u32(&sh.acc_full[tile & 1]), 1));
                    break;
                }
                mma_commit_pair(&sh.acc_full[tile & 1], (uint16_t)0x3);
            }
            sh.consumed = it;
        }
        __syncwarp();
    } else if (warp < 2 + kEpiWarps) {
        // ---- epilogue: TMEM lane quarter = warp % 4; four 32-column slices each, the shared columns first ----
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int row = quarter * 32 + lane;
        uint8_t *piece = sh.piece[warp - 2];
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t acc_shared = mapa_shared(smem_u32(&sh.acc_shared), 0);
        int tile = 0;
        for (int u = cl; u < units; u += ncl, ++tile) {
            int p0, q0;
            pair_coords(u, p_tiles, q_tiles, p0, q0);
            const int m = p0 + (int)rank * kHalf + row;
            const int second = tile & 1;
            // the first column of this warp's slice i: the shared columns (128-255 of the first accumulator,
            // 0-127 of the second) come first; slices 2i and 2i + 1 are neighbours
            auto column = [&](int i) {
                const int c = 128 * (i >> 1) + 64 * half + 32 * (i & 1);
                return second ? c : (c + kAcc1Col) & 255;
            };
            float lb[4];  // the tile's bias, one value per lane and slice, read while the MMAs run
#pragma unroll
            for (int i = 0; i < 4; ++i) lb[i] = bias_lane(bias, q0 + column(i), N);
            const bool ok = mbar_wait(&sh.acc_full[second], (tile >> 1) & 1, status, kSiteAccum);
            tc_fence_after();
            // warp-uniform, so that the bias shuffles below run on all 32 lanes
            const bool have = __all_sync(0xFFFFFFFFu, ok && !*((volatile int32_t *)&sh.aborted));
#pragma unroll
            for (int pair = 0; pair < 2; ++pair) {
                uint32_t p[32];  // 64 columns of this lane's row, in bf16
                const int n0 = q0 + column(2 * pair);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v[32];
                    if (have) {
                        uint32_t r0[16], r1[16];
                        const uint32_t at = lanes + (uint32_t)(second * kAcc1Col + n0 - q0 + 32 * i);
                        tmem_ld16(at, r0);
                        tmem_ld16(at + 16, r1);
                        tmem_ld_wait16(r0);
                        tmem_ld_wait16(r1);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            v[j] = __uint_as_float(r0[j]);
                            v[16 + j] = __uint_as_float(r1[j]);
                        }
                    }
                    if (pair == 0 && i == 1) {  // the shared columns are out
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(acc_shared);
                    }
                    if (!have) continue;
                    if (bias) bias_add32(v, pair ? lb[2 + i] : lb[i]);  // warp-uniform condition
#pragma unroll
                    for (int j = 0; j < 16; ++j) p[16 * i + j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                    if (ALIGNED && n0 + 32 * i < N) {  // warp-uniform
                        if (lane == 0) bulk_wait_read();  // the piece before has left shared memory
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 4; ++j)  // 16-byte unit j of the row, at j ^ (row / 2) % 4
                            *reinterpret_cast<uint4 *>(piece + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) =
                                make_uint4(p[16 * i + 4 * j], p[16 * i + 4 * j + 1], p[16 * i + 4 * j + 2],
                                           p[16 * i + 4 * j + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        // (rows and columns past the end are cut off)
                        if (lane == 0 && m < M) tma_store_2d(&tm_out, piece, n0 + 32 * i, m);
                    }
                }
                if (!ALIGNED && have && n0 < N) {
                    uint16_t *o = out + (size_t)(m - lane) * N + n0;
                    const int rows = M - (m - lane), cols = min(N - n0, 64);
                    if (N % 4 == 0)
                        store_rows<uint2, false>(o, piece, p, rows, cols, N, lane);
                    else if (N % 2 == 0)
                        store_rows<uint32_t, false>(o, piece, p, rows, cols, N, lane);
                    else
                        store_rows<uint32_t, true>(o, piece, p, rows, cols, N, lane);
                }
            }
            tc_fence_before();
            if (!have) break;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        // ---- scales ----
        const int st = tid - 32 * (2 + kEpiWarps);
        const int quarter = warp & 3;
        const uint32_t slot0 = tmem + (uint32_t)kSfCol + ((uint32_t)(quarter * 32) << 16);
        int step = 0;
        const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0);
        const uint8_t *xlo = xs, *xhi = xs + (size_t)M * nb, *wlo = ws, *whi = ws + (size_t)N * nb;
        const int D = (C + 1) / 2;  // steps of two chunks
        int it = 0;
        bool stop = false;
        for (int u = cl; u < units; u += ncl) {
            int p0, q0;
            pair_coords(u, p_tiles, q_tiles, p0, q0);
            const int ra = p0 + (int)rank * kHalf + 32 * quarter + lane, rb0 = q0 + st, rb1 = rb0 + kHalf;
            const bool ia = ra < M, ib0 = rb0 < N, ib1 = rb1 < N;
            const uint8_t *pa = xs + (size_t)(ia ? ra : 0) * nb, *pb0 = ws + (size_t)(ib0 ? rb0 : 0) * nb,
                          *pb1 = ws + (size_t)(ib1 ? rb1 : 0) * nb;
            // !SHIFTED: the 16-byte blocks of the next two steps, in registers
            const uint4 one = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            auto block = [&](const uint8_t *p, int k, bool in) {
                return in && 16 * k < nb ? __ldg(reinterpret_cast<const uint4 *>(p) + k) : one;
            };
            uint4 va[2], vb0[2], vb1[2];
            // SHIFTED: block k, counted from the 16-byte boundary before the row, on its way to shared memory.  A
            // step's bytes lie across two blocks; the three after its first are asked for before it starts.
            auto off = [](const uint8_t *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15u); };
            const int ma = off(pa), na = ia ? nb : 0, ka = ia ? (ma + nb + 15) / 16 : 0;  // place, bytes, blocks
            const int mb0 = off(pb0), nb0 = ib0 ? nb : 0, kb0 = ib0 ? (mb0 + nb + 15) / 16 : 0;
            const int mb1 = off(pb1), nb1 = ib1 ? nb : 0, kb1 = ib1 ? (mb1 + nb + 15) / 16 : 0;
            auto ask = [&](int k) {
                uint4(*to)[kHalf] = sh.raw[k % kRaw];
                if (k < ka) copy_block(&to[0][st], pa - ma + 16 * k, xlo, xhi);
                if (k < kb0) copy_block(&to[1][st], pb0 - mb0 + 16 * k, wlo, whi);
                if (k < kb1) copy_block(&to[2][st], pb1 - mb1 + 16 * k, wlo, whi);
                cp_async_commit();
            };
            auto take = [&](int r, int m, int n, int s) {  // the bytes of step s, 1.0 from byte n of the row on
                return scales_until(shift_blocks(sh.raw[s % kRaw][r][st], sh.raw[(s + 1) % kRaw][r][st], m),
                                    n - 16 * s);
            };
            if constexpr (SHIFTED) {
                for (int k = 0; k < kRaw - 1; ++k) ask(k);
            } else {
#pragma unroll
                for (int d = 0; d < 2; ++d)
                    va[d] = block(pa, d, ia), vb0[d] = block(pb0, d, ib0), vb1[d] = block(pb1, d, ib1);
            }
            // A warp that gave up goes on through the barriers, so that no other one waits for it there.
            for (int s2 = 0; s2 < D; ++s2, ++step) {
                uint4 *buf = sh.scales[step & 1], a;
                if constexpr (SHIFTED) {
                    ask(s2 + kRaw - 1);
                    cp_async_wait<kRaw - 2>();  // block s2 + 1 and those before it are there
                    a = take(0, ma, na, s2);
                    buf[st] = take(1, mb0, nb0, s2);
                    buf[kHalf + st] = take(2, mb1, nb1, s2);
                } else {
                    a = va[0];
                    buf[st] = vb0[0];
                    buf[kHalf + st] = vb1[0];
                    va[0] = va[1], vb0[0] = vb0[1], vb1[0] = vb1[1];
                    va[1] = block(pa, s2 + 2, ia), vb0[1] = block(pb0, s2 + 2, ib0), vb1[1] = block(pb1, s2 + 2, ib1);
                }
                // the buffer is whole; its last readers are past the barrier of the step before
                named_barrier(1, 32 * kScaleWarps);
                if (stop) continue;
                const int n = C - 2 * s2 < 2 ? 1 : 2;  // the step's chunks
                // their slots are free when the MMAs of the chunk kSlots before the last of them are done
                const int old = it + n - 1 - kSlots;
                if (old >= 0 && !mbar_wait(&sh.empty[old % kStages], (old / kStages) & 1, status, kSiteScale))
                    stop = true;
                if (__any_sync(0xFFFFFFFFu, stop || *((volatile int32_t *)&sh.aborted))) {
                    atomicExch(&sh.aborted, 1);
                    stop = true;
                    continue;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == n) break;
                    uint2 wb[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) wb[j] = reinterpret_cast<const uint2 *>(&buf[32 * j + lane])[h];
                    const uint32_t sf = slot0 + (uint32_t)(kSlotCols * ((it + h) % kSlots));
                    const uint32_t a0 = h ? a.z : a.x, a1 = h ? a.w : a.y;
                    tmem_st4(sf, a0, a0, a0, a0);  // column `quarter` of the four is the one read
                    tmem_st4(sf + 8, a1, a1, a1, a1);
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        tmem_st4(sf + 16 + j, wb[j].x, wb[j + 1].x, wb[j + 2].x, wb[j + 3].x);
                        tmem_st4(sf + 24 + j, wb[j].y, wb[j + 1].y, wb[j + 2].y, wb[j + 3].y);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane < n) mbar_arrive_remote(full0 + (uint32_t)(((it + lane) % kStages) * sizeof(uint64_t)));
                it += n;
            }
            if (SHIFTED) cp_async_wait<0>();  // the next tile's blocks go to the same places
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    // Drain TMA copies that were issued but never consumed (only after a timeout).
    if (tid == 0 && leader) {
        for (int i = sh.consumed; i < sh.issued; ++i)
            if (!mbar_wait(&sh.full[i % kStages], (i / kStages) & 1, status, kSiteDrain)) break;
    }
    // No remote arrival, copy or MMA operand read is left in flight past here.
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

constexpr int kMaxDevices = 64;
int g_clusters[kMaxDevices];  // co-resident clusters of 2, per device

template <bool SHIFTED>
constexpr int smem_bytes() {
    return 1024 + PairShared<SHIFTED>::kStages * kStageBytes + (int)sizeof(PairShared<SHIFTED>);
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory");
static_assert(smem_bytes<false>() > 116 * 1024 && smem_bytes<true>() > 116 * 1024,
              "one CTA per SM: each allocates all 512 TMEM columns");
int smem_of(bool shifted) { return shifted ? smem_bytes<true>() : smem_bytes<false>(); }

using PairFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const uint8_t *, const uint8_t *,
                        const uint16_t *, uint16_t *, int, int, int, int32_t *);

PairFn pick_pair(bool shifted, bool aligned) {
    if (shifted) return aligned ? mxfp4_pair_kernel<true, true> : mxfp4_pair_kernel<true, false>;
    return aligned ? mxfp4_pair_kernel<false, true> : mxfp4_pair_kernel<false, false>;
}

cudaLaunchConfig_t pair_config(int clusters, int smem, uint32_t flags, void *stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = (cudaStream_t)stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cfg;
}

}  // namespace

int init_mxfp4_pair() {
    for (bool shifted : {false, true})
        for (bool aligned : {false, true}) {
            const int e = (int)cudaFuncSetAttribute(pick_pair(shifted, aligned),
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(shifted));
            if (e) return e;
        }
    int dev = 0;
    const int e = (int)cudaGetDevice(&dev);
    if (e || dev < 0 || dev >= kMaxDevices) return e ? e : (int)cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pair_config(kGb300Sms, smem_of(false), 0, nullptr, attr);
    cfg.numAttrs = 1;
    int n = 0;
    // A failed query only loses the clamp (launches then use half the SMs' number).
    if (cudaOccupancyMaxActiveClusters(&n, pick_pair(false, true), &cfg) != cudaSuccess) {
        n = 0;
        (void)cudaGetLastError();
    }
    g_clusters[dev] = n;
    return 0;
}

float mxfp4_pair_estimate(int M, int N, int K, int num_sms) {
    // 0.42 us a chunk and round of tiles (K = 7168: 15.4 us for one round, 4096: 11, 1024: 5.4)
    const long long units = (long long)tiles_of(M) * tiles_of(N);
    const long long rounds = (units + num_sms / 2 - 1) / (num_sms / 2);
    return 0.42f * (float)chunks_of(K) * (float)rounds;
}

int launch_mxfp4_pair(const void *xq, const void *xs, const void *wq, const void *ws, const void *bias, void *out,
                      int M, int N, int K, int num_sms, uint32_t flags, void *stream, int32_t *status) {
    CUtensorMap tx, tw;  // 128-byte rows of 256 codes
    int r = make_tmap_u8_2d(&tx, xq, (uint64_t)M, (uint64_t)(K / 2), kHalf, kChunkBytes, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (r) return (int)cudaErrorInvalidValue;
    r = make_tmap_u8_2d(&tw, wq, (uint64_t)N, (uint64_t)(K / 2), kHalf, kChunkBytes, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (r) return (int)cudaErrorInvalidValue;
    CUtensorMap to = {};  // 32 x 32 pieces of out; not used where its rows are not 16-byte aligned
    if (N % 8 == 0) {
        r = make_tmap_bf16_2d(&to, out, (uint64_t)M, (uint64_t)N, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_NONE);
        if (r) return (int)cudaErrorInvalidValue;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return (int)cudaErrorInvalidDevice;
    // A cluster that cannot be resident with the others would run its tiles after them.
    const long long units = (long long)tiles_of(M) * tiles_of(N);
    long long clusters = g_clusters[dev] > 0 ? g_clusters[dev] : num_sms / 2;
    if (units < clusters) clusters = units;
    const uintptr_t a = reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(ws) | (uintptr_t)(K / 32);
    const bool shifted = a % 16 != 0;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = pair_config((int)clusters, smem_of(shifted), flags, stream, attr);
    return (int)cudaLaunchKernelEx(&cfg, pick_pair(shifted, N % 8 == 0), tx, tw, to, static_cast<const uint8_t *>(xs),
                                   static_cast<const uint8_t *>(ws), static_cast<const uint16_t *>(bias),
                                   static_cast<uint16_t *>(out), M, N, K, status);
}

}  // namespace bf16l
