// grouped.cu — out[p] = x[row of p] @ W[e]^T (+ bias[e]) for the rows p of each group e, their numbers known on the
// device alone; with SwiGLU, W[e] holds N gate rows and then N up rows and out = silu(gate) * up.
//
// W rows on the MMA's M side and rows of x on its N side, by CTA pairs (cta_group::2): a tile is 256 W rows (128 of each
// CTA) by up to `bt` rows of one group.  A group has few rows or many, and an MMA's time goes with its N: so a group's rows
// are split evenly over as few tiles as hold them, and each tile's MMAs take its own N, a multiple of 32.  A weight is read
// for each of its group's row tiles, one after the other, so once from HBM.
//
//   * every CTA turns the offsets into the first tile of each group (a scan in shared memory) and each role finds a tile's
//     group by bisection;
//   * warp 0: TMA producer: two chunks of 128 bytes of K a stage of this CTA's own W rows (a 4-D map: a row past the
//     group's weight is zero, not the next group's) and of its half of the tile's rows of x, by boxes of 16 to 128 rows;
//   * warps 10-13, where `rows` gives the rows of x: 16-byte asynchronous copies from where they are, so that no sorted copy
//     of x is made; they arrive by themselves on a barrier of the CTA, and warp 14 passes that on to the leader's.  (TMA's
//     gather of four rows an instruction takes about 12 clocks a row, three times what a stage of MMAs leaves: 8192 rows of 8
//     choices, 128 groups, 2 x 2048 x 7168: 9.05 ms, 2.5 so.);
//   * warp 1 of the even CTA: MMA issuer; warps 2-9: epilogue, two for each quarter of the TMEM lanes;
//   * fp32 accumulators double-buffered in TMEM;
//   * SwiGLU: boxes of 16 gate rows and their 16 up rows, so that a warp's 32 lanes hold both: one shuffle for two rows
//     of x brings them together in fp32, and out is written without the wide product's way through memory.
// The same kernel runs the two products of a linear's adapters for many rows, ordered by adapter (rows of none last):
//   * kInner: h = scale_e * x @ A_e^T, the groups being the adapters; out is the value's first eight bits and the rest, rounded
//     to eight bits, so that the tensor cores take 16 bits of it;
//   * kOuter: x @ W^T with 256 rows of x on the M side and 256 W rows on the N side, whose tiles then go on along K with the
//     adapters that their rows have: 16 ranks a slot, eight slots a stage, each slot a tile of B_e (16 columns, 32-byte
//     swizzle) against the rows' h, its MMAs writing the TMEM lanes of that adapter's rows alone (the MMA's lane mask), so
//     that nothing of one adapter, not finite or not, reaches a row of another.  A row of out is written where its row of
//     x is.
// Where the tiles are too few for the SMs (PARTIAL), each tile's K is split into parts of their own tiles, which leave their
// fp32 accumulators in a workspace, and sum_kernel adds them up in order.
// What bounds it: with a few rows a group HBM, every sought weight being read once (512 rows over 101 weights of 7168 x 2048
// 425 us, 8 rows over 8 of 2 x 2048 x 7168 72 us: 102% and 96% of the copy rate); with hundreds of rows a group the tensor
// cores: 1.74 to 1.84 PFLOP/s over one to eight groups while the clock holds, 1.6 at the 1.46 GHz that the power limit leaves.
// 128 uneven groups (65536 rows) take 17% more clocks than even ones of 512: their tiles have 202 rows on average, and every
// tile takes all of its W rows in (a tile of 160 rows 85% of the time of one of 256).
// Cross-CTA lifetime: a cluster barrier after set-up (every barrier exists before any remote arrival or copy) and one
// before TMEM is freed and the CTAs exit.  Every wait is bounded.
#include <cuda_runtime.h>

#include "grouped.cuh"
#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

constexpr int kHalf = 128;                        // W rows per CTA
constexpr int kWBytes = kHalf * kChunkK * 2;      // of a stage
constexpr int kChunks = 2;  // 64-wide chunks of K in a stage
constexpr int kMaxStages = 8;
constexpr int kEpiWarps = 8;
constexpr int kGatherWarps = 4, kGatherRows = 4 * kGatherWarps;  // (a warp copies four rows' 128 bytes at a time)
__host__ __device__ constexpr int threads_of(bool gather) { return 32 * (2 + kEpiWarps + (gather ? kGatherWarps + 1 : 0)); }
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kPer = (kMaxGroups + 32 * (2 + kEpiWarps) - 1) / (32 * (2 + kEpiWarps));  // groups of a thread, at most
constexpr int kRank = 16, kSlots = 2 * kChunkK / kRank;  // ranks of a slot, slots of a stage
constexpr int kPiece = 32, kPieceBytes = 32 * kPiece * 2;  // kOuter: columns of out that a warp gathers before it stores them

enum Mode { kPlain, kSwiglu, kInner, kOuter };
// W rows of a CTA and chunk have this much of a stage: kInner's are at most 64 (the MMA's other rows are whatever follows,
// and so are their lanes of the accumulator, which nobody reads).
__host__ __device__ constexpr int w_bytes(int mode) { return mode == kInner ? kWBytes / 2 : kWBytes; }

struct GroupedShared {
    uint8_t piece[kEpiWarps][kPieceBytes];  // kOuter
    uint64_t full[kMaxStages];   // leader only: both CTAs' copies of the stage have landed
    uint64_t empty[kMaxStages];  // both: the MMAs reading the stage are done
    uint64_t copied[kMaxStages]; // this CTA's rows of x by index are in shared memory
    uint64_t acc_full[2];        // both: the accumulator holds a finished tile
    uint64_t acc_empty[2];       // leader only: both CTAs' epilogues have read it
    uint32_t off[kSlots][8];  // kOuter: the lane masks of a stage's slots
    int32_t column[kSlots];   // ... and their places in a row of h, in 16 bytes
    uint32_t tmem_base;
    int32_t bad_pair, aborted, issued, consumed;
    int32_t part[2][threads_of(true) / 32];
    int32_t tiles[kMaxGroups + 1];  // row tiles before each group
    int32_t first[kMaxGroups + 1];  // first row of each group; kOuter: of each adapter that has rows, then of the rows of none
    int32_t count[kMaxGroups];      // its rows; kOuter: which adapter
};

// Unit u: a row tile of a group and 256 W rows (128 outputs with SwiGLU); row tiles vary fastest.
struct Unit {
    int e, p0, rows, m;  // group, first position, rows, W tile
    int cols;            // rows rounded up for the MMA
    int part, c0, n;     // PARTIAL: which part of K; its first stage, and its stages
};
// a / b of what nearly always fits 32 bits (a 64-bit division is a long routine, and the first load waits for this one).
__device__ __forceinline__ int quotient(long long a, int b) {
    return a >> 32 ? (int)(a / b) : (int)((uint32_t)a / (uint32_t)b);
}
// ONE: a single group of n rows, in whole tiles of bt; else n groups.
template <bool ONE>
__device__ __forceinline__ Unit unit_of(const GroupedShared &sh, int n, int bt, long long u, int m_tiles) {
    int lo = 0, hi = ONE ? 1 : n;  // tiles[lo] <= q < tiles[hi]
    const int q = m_tiles == 1 ? (int)u : quotient(u, m_tiles);
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh.tiles[mid] <= q)
            lo = mid;
        else
            hi = mid;
    }
    const int before = ONE ? 0 : sh.tiles[lo];
    const int nt = ONE ? (n + bt - 1) / bt : sh.tiles[lo + 1] - before, count = ONE ? n : sh.count[lo];
    const long long local = u - (long long)before * m_tiles;
    const int m = nt == 1 ? (int)local : quotient(local, nt), t = (int)(local - (long long)m * nt);
    const int each = nt == 1 ? count : count / nt, more = count - each * nt;
    Unit r;
    r.e = lo;
    r.m = m;
    r.rows = ONE ? min(bt, n - t * bt) : each + (t < more);
    r.p0 = ONE ? t * bt : sh.first[lo] + t * each + min(t, more);
    r.cols = ONE ? bt : (r.rows + 31) & ~31;
    return r;
}

// kOuter: the adapters of a tile's rows (of those that have rows), and the stages that they add: for each 64 ranks, slots of
// 16 for one adapter after the other.
struct Tail {
    int first, n, R;
    __device__ __forceinline__ int per(int kb) const { return (min(R - kb * kChunkK, kChunkK) + kRank - 1) / kRank; }
    __device__ __forceinline__ int stages_of(int kb) const { return (n * per(kb) + kSlots - 1) / kSlots; }
    __device__ __forceinline__ int stages() const { return n ? stages_of(0) + (R > kChunkK ? stages_of(1) : 0) : 0; }
};
struct TailStage {
    int kb, per, q0, n;  // block of 64 ranks, slots of an adapter in it, first slot, slots
};
__device__ __forceinline__ TailStage tail_stage(const Tail &f, int d) {
    const int s0 = f.stages_of(0);
    TailStage r;
    r.kb = d >= s0;
    r.per = f.per(r.kb);
    r.q0 = (d - (r.kb ? s0 : 0)) * kSlots;
    r.n = min(kSlots, f.n * r.per - r.q0);
    return r;
}
__device__ __forceinline__ Tail tail_of(const GroupedShared &sh, int adapters, const Unit &t, int R) {
    auto below = [&](int p) {  // adapters (and the rows of none) that start below position p
        int lo = 0, hi = adapters + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sh.first[mid] < p)
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo;
    };
    Tail r;
    r.R = R;
    r.first = max(below(t.p0 + 1) - 1, 0);
    r.n = max(min(below(t.p0 + t.rows), adapters) - r.first, 0);
    return r;
}
// A word of the MMA's lane mask: bits lo .. hi - 1 (of 0 .. 31) clear, those rows to be written.
__device__ __forceinline__ uint32_t lanes_but(int lo, int hi) {
    const int l = min(max(lo, 0), 32), h = min(max(hi, 0), 32);
    return ~((h < 32 ? (1u << h) - 1u : ~0u) & ~(l < 32 ? (1u << l) - 1u : ~0u));
}

// A role's place in the ring.  (A stage's number divided by the runtime ring depth costs each role some 250 clocks a stage.)
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) s = 0, phase ^= 1;
    }
};

// Whether `n` rows from position q on are neighbours in x (the whole warp asks).
__device__ __forceinline__ bool neighbours(const int32_t *rows, int q, int n, int x_rows) {
    const int lane = threadIdx.x & 31, first = __ldg(rows + q);
    bool ok = first >= 0 && first <= x_rows - n;
    for (int i = lane; i < n; i += 32) ok = ok && __ldg(rows + q + i) == first + i;
    return __all_sync(kAll, ok);
}

// Maps of x with boxes of 16, 32, 64 and 128 rows.
struct RowMaps {
    CUtensorMap of[4];
};

template <int BYTES>
struct Word;
template <>
struct Word<16> {
    using T = uint4;
};
template <>
struct Word<8> {
    using T = uint2;
};
template <>
struct Word<4> {
    using T = uint32_t;
};
template <>
struct Word<2> {
    using T = uint16_t;
};
// A piece of 32 rows by kPiece columns (16-byte unit j of row r at j ^ (r / 2) % 4) to rows of out, BYTES a lane: `rows` of
// them (lane r's `to` is the row that r goes to), `cols` columns, a multiple of BYTES' elements.
template <int BYTES>
__device__ __forceinline__ void store_piece(uint16_t *out, const uint8_t *piece, int to, int rows, int cols, int N, int lane) {
    using T = typename Word<BYTES>::T;
    constexpr int lanes = 2 * kPiece / BYTES;  // of a row
    const int r0 = lane / lanes, byte = lane % lanes * BYTES;
#pragma unroll
    for (int k = 0; k < 32; k += 32 / lanes) {
        const int r = k + r0, row = __shfl_sync(kAll, to, r);
        const T w = *reinterpret_cast<const T *>(piece + 64 * r + ((byte & ~15) ^ (((r >> 1) & 3) << 4)) + (byte & 15));
        if (r < rows && byte < 2 * cols) *reinterpret_cast<T *>(out + (size_t)row * N + byte / 2) = w;
    }
}

template <int MODE, bool GATHER, bool PARTIAL>
__global__ void __launch_bounds__(threads_of(GATHER), 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_b,
                   const __grid_constant__ RowMaps tm_x, const GroupedArgs a,
                   int w_boxes, int bt, int wt, int stages, int32_t *status) {
    constexpr bool SWIGLU = MODE == kSwiglu;
    static_assert(GATHER || MODE == kPlain || MODE == kSwiglu, "the adapters' rows go by index");
    constexpr int kThreads = threads_of(GATHER);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    constexpr int kWSpace = w_bytes(MODE);
    const int chunk_bytes = kWSpace + bt * kChunkK;  // W rows, and bt / 2 rows of x, of 128 bytes
    const int stage_bytes = kChunks * chunk_bytes;
    constexpr int kW = MODE == kOuter ? kWBytes : 0, kX = MODE == kOuter ? 0 : kWSpace;  // (the M side's rows first)
    GroupedShared &sh = *reinterpret_cast<GroupedShared *>(ring + stages * stage_bytes);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    // wt: outputs of a W tile, half of them a CTA's (kInner: of its W rows, so that both CTAs have some)
    const int m_tiles = (a.N + wt - 1) / wt;
    const uint32_t w_chunk = MODE == kInner || MODE == kOuter ? (uint32_t)wt * kChunkK : (uint32_t)kWBytes;  // bytes of a box
    const int cl = (int)blockIdx.x >> 1, ncl = (int)gridDim.x >> 1;
    const int C = (a.K + kChunkK * kChunks - 1) / (kChunkK * kChunks);  // stages of a tile (zeros past K)
    const uint32_t tmem_cols = 2u * (uint32_t)bt;
    const int slot_bytes = wt * kRank;  // kOuter: 16 ranks of this CTA's wt / 2 rows of B

    if (tid == 0) {
        tma_prefetch_desc(&tm_w);
        if (!GATHER)
            for (int i = 0; i < 4; ++i) tma_prefetch_desc(&tm_x.of[i]);
        if (MODE == kOuter) tma_prefetch_desc(&tm_x.of[3]);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&sh.full[s], GATHER ? 3 : 1);  // the leader producer's arrive.expect_tx, each CTA's copies of x
            mbar_init(&sh.copied[s], 32 * kGatherWarps);
            mbar_init(&sh.empty[s], 1);  // the leader's multicast commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], 2 * kEpiWarps);
        }
        sh.aborted = 0;
        sh.issued = 0;
        sh.consumed = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&sh.tmem_base, tmem_cols);
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
    pdl_launch_dependents();
    pdl_wait();  // nothing is read before the previous kernel has finished

    // `per` consecutive groups a thread.  First the offsets, made to rise (the largest of those before, over the block) ...
    const int per = (a.groups + kThreads - 1) / kThreads, e0 = min(tid * per, a.groups), e1 = min(e0 + per, a.groups);
    int end[kPer + 1];  // clamped offsets of this thread's groups
    int most = 0;
#pragma unroll
    for (int i = 0; i <= kPer; ++i) {
        end[i] = e0 + i <= e1 ? min(max(__ldg(a.offsets + e0 + i), 0), a.P) : 0;
        if (e0 + i < e1) most = max(most, end[i]);
    }
    int upto = most;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto = max(upto, v);
    }
    if (lane == 31) sh.part[0][warp] = upto;
    upto = __shfl_up_sync(kAll, upto, 1);
    __syncthreads();
    int before = lane ? upto : 0;
    for (int w = 0; w < warp; ++w) before = max(before, sh.part[0][w]);
#pragma unroll
    for (int i = 0; i <= kPer; ++i) before = end[i] = max(before, end[i]);
    // ... then the row tiles before each group (kOuter: the adapters that have rows).
    auto weight = [&](int i) {
        const int n = end[i + 1] - end[i];
        return MODE == kOuter ? (n > 0 ? 1 : 0) : (n + bt - 1) / bt;
    };
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (e0 + i < e1) mine += weight(i);
    upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 31) sh.part[1][warp] = upto;
    __syncthreads();
    before = upto - mine;
    for (int w = 0; w < warp; ++w) before += sh.part[1][w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (e0 + i >= e1) continue;
        const int n = weight(i);
        if (MODE != kOuter) {
            sh.tiles[e0 + i] = before;
            sh.first[e0 + i] = end[i];
            sh.count[e0 + i] = end[i + 1] - end[i];
        } else if (n) {
            sh.first[before] = end[i];
            sh.count[before] = e0 + i;
        }
        before += n;
        if (e0 + i + 1 == a.groups) {
            sh.tiles[MODE == kOuter ? 0 : a.groups] = before;
            if (MODE == kOuter) sh.first[before] = end[i + 1];
        }
    }
    __syncthreads();
    const bool bad_pair = sh.bad_pair != 0;  // the same verdict in both CTAs
    const int adapters = MODE == kOuter ? sh.tiles[0] : 0;
    const long long units = (long long)(MODE == kOuter ? (a.P + bt - 1) / bt : sh.tiles[a.groups]) * m_tiles *
                            (PARTIAL ? a.splits : 1);
    auto unit = [&](long long u) {
        const int s = PARTIAL ? (int)(u % a.splits) : 0;
        Unit t = unit_of<MODE == kOuter>(sh, MODE == kOuter ? a.P : a.groups, bt, PARTIAL ? u / a.splits : u, m_tiles);
        t.part = s;
        t.c0 = PARTIAL ? C * s / a.splits : 0;
        t.n = PARTIAL ? C * (s + 1) / a.splits - t.c0 : C;
        return t;
    };
    auto tail = [&](const Unit &t) {  // (with the last part of K)
        return MODE == kOuter && (!PARTIAL || t.part == a.splits - 1) ? tail_of(sh, adapters, t, a.R) : Tail{0, 0, 0};
    };

    if (bad_pair) {
        // nothing issued: fall through to the exit barrier
    } else if (warp == 0) {
        // ---- TMA producer (both CTAs): the whole warp goes through the loop, one elected lane issues ----
        const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0);  // leader's full[0]
        int it = 0;
        Ring r;
        bool ok = true;
        for (long long u = cl; ok && u < units; u += ncl) {
            const Unit t = unit(u);
            const int half = t.cols >> 1, q0 = t.p0 + (int)rank * half;  // this CTA's rows of x
            const int n0 = t.m * wt + (int)rank * (wt / 2);
            const Tail f = tail(t);
            // kOuter: whole halves of neighbouring rows come by TMA
            bool near = false, near_other = false;
            int near_row = 0;
            if (MODE == kOuter) {
                near = t.p0 + t.rows >= q0 + kHalf && neighbours(a.rows, q0, kHalf, a.x_rows);
                const int other = t.p0 + (int)(rank ^ 1u) * kHalf;
                near_other = leader && t.p0 + t.rows >= other + kHalf && neighbours(a.rows, other, kHalf, a.x_rows);
                near_row = near ? __ldg(a.rows + q0) : 0;
            }
            for (int c = 0, n = t.n + f.stages(); c < n; ++c, ++it, r.next(stages)) {
                const int s = r.s;
                ok = mbar_wait(&sh.empty[s], r.phase ^ 1u, status, kSiteEmpty);  // (at once in the first round)
                ok = __all_sync(kAll, ok && !*((volatile int32_t *)&sh.aborted));
                if (!ok) {
                    if (lane == 0) atomicExch(&sh.aborted, 1);
                    break;
                }
                uint8_t *st = ring + s * stage_bytes;
                const uint32_t fb = full0 + (uint32_t)(s * sizeof(uint64_t));
                if (elect_one()) {
                    if (MODE == kOuter && c >= t.n) {  // tiles of B
                        const TailStage g = tail_stage(f, c - t.n);
                        if (leader) mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(2 * g.n * slot_bytes));
                        int i = f.first + g.q0 / g.per, b16 = g.q0 % g.per;
                        for (int j = 0; j < g.n; ++j) {
                            tma_load_4d_pair(st + (j >> 2) * chunk_bytes + kW + (j & 3) * slot_bytes, &tm_b, fb,
                                             g.kb * kChunkK + b16 * kRank, n0, 0, sh.count[i]);
                            if (++b16 == g.per) b16 = 0, ++i;
                        }
                    } else {
                        if (leader) {
                            const uint32_t x_bytes = GATHER ? (uint32_t)(near + near_other) * kHalf * kChunkK * 2
                                                            : (uint32_t)(t.cols * kChunkK * 2);
                            mbar_arrive_expect_tx(&sh.full[s], (uint32_t)kChunks * (2u * w_chunk + x_bytes));
                        }
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            const int k0 = ((t.c0 + c) * kChunks + j) * kChunkK;
                            uint8_t *ch = st + j * chunk_bytes;
                            if (!SWIGLU) {
                                tma_load_4d_pair(ch + kW, &tm_w, fb, k0, n0, 0, t.e);
                            } else if (w_boxes == 1) {
                                tma_load_5d_pair(ch, &tm_w, fb, k0, 0, 0, n0 >> 4, t.e);
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    tma_load_4d_pair(ch + i * (kWBytes / 4), &tm_w, fb, k0, n0 + 16 * i, 0, t.e);
                            }
                            if (MODE == kOuter && near) tma_load_2d_pair(ch + kX, &tm_x.of[3], fb, k0, near_row);
                            // this CTA's rows, a multiple of 16, by boxes of falling sizes
#pragma unroll
                            for (int i = 3; i >= 0; --i)
                                if (!GATHER && (half & (16 << i))) {
                                    const int first = half & ~((32 << i) - 1);
                                    tma_load_2d_pair(ch + kX + first * 128, &tm_x.of[i], fb, k0, q0 + first);
                                }
                        }
                    }
                }
            }
        }
        if (lane == 0) sh.issued = it;
        // Every commit that arrives on this CTA's `empty` barriers has landed before the exit barrier.
        if (ok) {
            for (int i = 0; i < stages; ++i, r.next(stages))
                if (!mbar_wait(&sh.empty[r.s], r.phase ^ 1u, status, kSiteDrain)) break;
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (leader only): the whole warp goes through the loop and one elected lane issues, so that descriptors
        // are uniform (8 MMAs and a commit 196 clocks; by lane 0 in a branch of its own 555) ----
        if (leader) {
            int it = 0, tile = 0;
            Ring r;
            bool ok = true;
            const uint32_t first_lo = (uint32_t)smem_desc_sw128(smem_u32(ring));  // (the low word)
            for (long long u = cl; ok && u < units; u += ncl, ++tile) {
                const Unit t = unit(u);
                const Tail f = tail(t);
                const uint32_t idesc = idesc_bf16_f32(2 * kHalf, MODE == kOuter ? wt : t.cols);
                const int b = tile & 1, n = t.n + f.stages();
                const uint32_t acc = tmem + (uint32_t)(b * bt);
                if (lane == 0) sh.consumed = it;
                // Both CTAs' epilogues have read this buffer (used two tiles ago).
                ok = __all_sync(kAll, tile < 2 || mbar_wait(&sh.acc_empty[b], ((tile >> 1) - 1) & 1, status, kSiteTmemEmpty));
                tc_fence_after();
                for (int c = 0; ok && c < t.n; ++c, ++it, r.next(stages)) {
                    const int s = r.s;
                    ok = __all_sync(kAll, mbar_wait(&sh.full[s], r.phase, status, kSiteFull));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t lo = first_lo + (uint32_t)s * (uint32_t)(stage_bytes >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            const uint32_t alo = lo + j * (uint32_t)(chunk_bytes >> 4);
#pragma unroll
                            for (int kk = 0; kk < kChunkK / 16; ++kk)
                                mma_bf16_pair_sw128(acc, alo + 2 * kk, alo + ((MODE == kOuter ? kW : kX) >> 4) + 2 * kk, idesc,
                                                    j + kk > 0 ? 1u : (uint32_t)c);
                        }
                        mma_commit_pair(&sh.empty[s], (uint16_t)0x3);
                    }
                }
                if (MODE == kOuter) {
                    for (int c = t.n; ok && c < n; ++c, ++it, r.next(stages)) {
                        // Four lanes a slot: its MMAs' lane mask and its place in h, which one lane would take longer
                        // to work out than the MMAs take.
                        const TailStage g = tail_stage(f, c - t.n);
                        const int q = g.q0 + (lane >> 2), i = f.first + q / g.per, w = 2 * (lane & 3);
                        if ((lane >> 2) < g.n) {
                            const int lo = sh.first[i] - t.p0, hi = min(sh.first[i + 1] - t.p0, t.rows);
                            sh.off[lane >> 2][w] = lanes_but(lo - 32 * w, hi - 32 * w);
                            sh.off[lane >> 2][w + 1] = lanes_but(lo - 32 * w - 32, hi - 32 * w - 32);
                            if (w == 0) sh.column[lane >> 2] = 2 * (q % g.per);
                        }
                        __syncwarp();
                        const int s = r.s;
                        if (elect_one()) {
                            ok = mbar_wait(&sh.full[s], r.phase, status, kSiteFull);
                            tc_fence_after();
                            const uint8_t *ch = ring + s * stage_bytes;
                            const uint32_t high = first_lo + (uint32_t)s * (uint32_t)(stage_bytes >> 4);
                            const uint32_t low = high + (uint32_t)(chunk_bytes >> 4);
                            uint32_t off[8];
                            int col = sh.column[0];
#pragma unroll
                            for (int w = 0; w < 8; ++w) off[w] = sh.off[0][w];
                            for (int j = 0; ok && j < g.n; ++j) {
                                const uint64_t bdesc =
                                    smem_desc_sw32(smem_u32(ch + (j >> 2) * chunk_bytes + kW + (j & 3) * slot_bytes));
                                // the next slot's, while this one's instructions go out
                                const int next = min(j + 1, kSlots - 1), col2 = sh.column[next];
                                uint32_t off2[8];
#pragma unroll
                                for (int w = 0; w < 8; ++w) off2[w] = sh.off[next][w];
                                mma_bf16_pair_lanes2(acc, high + (uint32_t)col, low + (uint32_t)col, bdesc, idesc, off);
                                col = col2;
#pragma unroll
                                for (int w = 0; w < 8; ++w) off[w] = off2[w];
                            }
                            if (ok) mma_commit_pair(&sh.empty[s], (uint16_t)0x3);
                        }
                        ok = __all_sync(kAll, ok);  // (the masks have been read)
                        if (!ok) break;
                    }
                }
                if (elect_one()) {
                    if (ok) {
                        mma_commit_pair(&sh.acc_full[b], (uint16_t)0x3);
                    } else {  // release both epilogues at once
                        atomicExch(&sh.aborted, 1);
                        sh.consumed = it;
                        mbar_arrive(&sh.acc_full[b]);
                        mbar_arrive_cluster(mapa_shared(smem_u32(&sh.acc_full[b]), 1));
                    }
                }
            }
            if (lane == 0) sh.consumed = it;
        }
        __syncwarp();
    } else if (GATHER && warp == 2 + kEpiWarps + kGatherWarps) {
        if (lane == 0) {  // ---- x by index: what has arrived, to the leader's barrier (both CTAs) ----
            const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0);
            Ring r;
            bool ok = true;
            for (long long u = cl; ok && u < units; u += ncl) {
                const Unit t = unit(u);
                const int n = t.n + tail(t).stages();
                for (int c = 0; ok && c < n; ++c, r.next(stages)) {
                    ok = mbar_wait(&sh.copied[r.s], r.phase, status, kSiteStage);
                    fence_proxy_async_smem();  // the copies, seen here, before the MMAs' reads
                    if (ok) mbar_arrive_remote(full0 + (uint32_t)(r.s * sizeof(uint64_t)));
                }
            }
            if (!ok) atomicExch(&sh.aborted, 1);
        }
        __syncwarp();
    } else if (GATHER && warp >= 2 + kEpiWarps) {
        // ---- x by index (both CTAs): eight lanes a row, kGatherRows rows at a time over the warps ----
        const int gt = tid - 32 * (2 + kEpiWarps), r0 = gt >> 3, v = gt & 7;
        const uint16_t *x = static_cast<const uint16_t *>(a.x) + 8 * v;
        const uint32_t to0 = smem_u32(ring) + kX + (uint32_t)(r0 * 128 + ((v ^ (r0 & 7)) << 4));
        Ring r;
        bool ok = true;
        for (long long u = cl; ok && u < units; u += ncl) {
            const Unit t = unit(u);
            const int half = t.cols >> 1, q0 = t.p0 + (int)rank * half;
            // Rows past the tile's are zero: one row read again by every CTA in their place is a hot spot (128 rows of
            // 14336 x 4096 with adapters: 74 us for the shared product alone, 44 so).
            const int have = min(max(t.p0 + t.rows - q0, 0), half);
            const bool near = MODE == kOuter && have == kHalf && neighbours(a.rows, q0, kHalf, a.x_rows);  // (they come by TMA)
            const uint16_t *row[kHalf / kGatherRows];
#pragma unroll
            for (int i = 0; i < kHalf / kGatherRows; ++i) {
                const int p = min(q0 + r0 + kGatherRows * i, t.p0 + t.rows - 1);
                row[i] = x + (size_t)min(max(__ldg(a.rows + p), 0), a.x_rows - 1) * a.K;
            }
            const Tail f = tail(t);
            for (int c = 0, n = t.n + f.stages(); c < n; ++c, r.next(stages)) {
                const int s = r.s;
                ok = mbar_wait(&sh.empty[s], r.phase ^ 1u, status, kSiteEmpty);
                ok = __all_sync(kAll, ok && !*((volatile int32_t *)&sh.aborted));
                if (!ok) {
                    if (lane == 0) atomicExch(&sh.aborted, 1);
                    break;
                }
                const uint32_t to = to0 + (uint32_t)(s * stage_bytes);
                if (MODE == kOuter && c >= t.n) {
                    // The rows' h: values, then remainders.
                    const int col = tail_stage(f, c - t.n).kb * kChunkK + 8 * v;
                    const uint16_t *h = static_cast<const uint16_t *>(a.h);
#pragma unroll 4
                    for (int i = 0; i < kHalf / kGatherRows; ++i) {
                        const int p = q0 + r0 + kGatherRows * i;
                        const bool in = col < a.R && p < t.p0 + t.rows;
                        const uint16_t *from = in ? h + (size_t)__ldg(a.rows + p) * 2 * a.R + col : h;
                        cp_async_16(to + 128 * kGatherRows * i, from, in ? 16u : 0u);
                        cp_async_16(to + (uint32_t)chunk_bytes + 128 * kGatherRows * i, in ? from + a.R : h, in ? 16u : 0u);
                    }
                    cp_async_arrive(&sh.copied[s]);
                    continue;
                }
                // The copies' own instructions count: four warps issue 16 each a stage, and one address serves all chunks.
                const int k0 = (t.c0 + c) * kChunks * kChunkK;
                if (near) {
                } else if (have == half && k0 + kChunks * kChunkK <= a.K) {
#pragma unroll
                    for (int i = 0; i < kHalf / kGatherRows; ++i)
                        if (kGatherRows * i < half) {
#pragma unroll
                            for (int j = 0; j < kChunks; ++j)
                                cp_async_16(to + j * (uint32_t)chunk_bytes + 128 * kGatherRows * i, row[i] + k0 + j * kChunkK);
                        }
                } else {
                    uint32_t in[kChunks];
#pragma unroll
                    for (int j = 0; j < kChunks; ++j) in[j] = k0 + j * kChunkK + 8 * v < a.K ? 16u : 0u;  // (K % 8 == 0)
#pragma unroll
                    for (int i = 0; i < kHalf / kGatherRows; ++i)
                        if (kGatherRows * i < half) {
                            const bool mine = r0 + kGatherRows * i < have;
#pragma unroll
                            for (int j = 0; j < kChunks; ++j)
                                cp_async_16(to + j * (uint32_t)chunk_bytes + 128 * kGatherRows * i,
                                            row[i] + (in[j] ? k0 + j * kChunkK : 0), mine ? in[j] : 0u);
                        }
                }
                cp_async_arrive(&sh.copied[s]);
            }
        }
        cp_async_wait_all();
        __syncwarp();
    } else {
        // ---- epilogue: TMEM lane quarter = warp % 4; the quarter's two warps take 16 rows of x in turn ----
        const int quarter = warp & 3, h = (warp - 2) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t acc_empty0 = mapa_shared(smem_u32(&sh.acc_empty[0]), 0);
        uint16_t *out = static_cast<uint16_t *>(a.out);
        const uint16_t *bias = static_cast<const uint16_t *>(a.bias);
        int tile = 0;
        for (long long u = cl; u < units; u += ncl, ++tile) {
            const Unit t = unit(u);
            const int b = tile & 1;
            // this lane's output, and the W row that it is of
            const int in_tile = SWIGLU ? quarter * 16 + (lane & 15) : quarter * 32 + lane;
            const int n = MODE == kInner && in_tile >= wt / 2 ? a.N : t.m * wt + (int)rank * (wt / 2) + in_tile;
            const int wide = SWIGLU ? 2 * a.N : a.N, wrow = SWIGLU && lane >= 16 ? a.N + n : n;
            const float f = MODE == kInner && a.scale ? __ldg(a.scale + t.e) : 1.0f;
            const bool biased = MODE != kOuter && bias && n < a.N && (!PARTIAL || t.part == 0);
            const float lb = biased ? bf16_to_f32(__ldg(bias + (size_t)t.e * wide + wrow)) : 0.0f;
            const bool ok = mbar_wait(&sh.acc_full[b], (tile >> 1) & 1, status, kSiteAccum);
            tc_fence_after();
            const bool have = __all_sync(kAll, ok && !*((volatile int32_t *)&sh.aborted));
            const uint32_t acc = lanes + (uint32_t)(b * bt);
            const bool pairs = (a.N & 1) == 0;
            if constexpr (MODE == kOuter) {  // this lane's row of x, kPiece outputs at a time
                const int i0 = (int)rank * kHalf + quarter * 32, left = t.rows - i0;  // the warp's first row, its rows
                uint8_t *piece = sh.piece[warp - 2];
                const int to = lane < left ? __ldg(a.rows + t.p0 + i0 + lane) : 0;
                for (int c0 = kPiece * h; have && c0 < wt && t.m * wt + c0 < a.N; c0 += 2 * kPiece) {
                    const int n0 = t.m * wt + c0;
                    const float nb = bias_lane(bias, n0, a.N);
                    uint32_t r0[16], r1[16];
                    tmem_ld16(acc + (uint32_t)c0, r0);
                    tmem_ld16(acc + (uint32_t)(c0 + 16), r1);
                    tmem_ld_wait16(r0);
                    tmem_ld_wait16(r1);
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[j] = __uint_as_float(r0[j]);
                        v[16 + j] = __uint_as_float(r1[j]);
                    }
                    if (bias && (!PARTIAL || t.part == 0)) bias_add32(v, nb);
                    if constexpr (PARTIAL) {
                        float *o = a.sums + ((size_t)t.part * a.P + to) * sum_pitch(a.N) + n0;
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            if (lane < left && n0 + j < a.N) OutStore<float>::eight(o + j, v + j);
                        __syncwarp();
                        continue;
                    }
                    __syncwarp();  // the piece before has been read
#pragma unroll
                    for (int j = 0; j < 4; ++j)  // 16-byte unit j of the row, at j ^ (row / 2) % 4
                        *reinterpret_cast<uint4 *>(piece + 64 * lane + 16 * (j ^ ((lane >> 1) & 3))) =
                            make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                       pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
                    __syncwarp();
                    // Neighbouring lanes store a row's 64 bytes, as wide as rows of N start (a row a lane: 8192 x 7168 x
                    // 7168 35 us more).
                    const int cols = min(a.N - n0, kPiece);
                    if (a.N % 8 == 0)
                        store_piece<16>(out + n0, piece, to, left, cols, a.N, lane);
                    else if (a.N % 4 == 0)
                        store_piece<8>(out + n0, piece, to, left, cols, a.N, lane);
                    else if (a.N % 2 == 0)
                        store_piece<4>(out + n0, piece, to, left, cols, a.N, lane);
                    else
                        store_piece<2>(out + n0, piece, to, left, cols, a.N, lane);
                }
            }
            // (a warp whose outputs all lie past N has nothing to do)
            const bool any = __any_sync(kAll, n < a.N);
            for (int c0 = 16 * h; MODE != kOuter && have && any && c0 < t.rows; c0 += 32) {
                uint32_t r[16];
                tmem_ld16(acc + (uint32_t)c0, r);
                tmem_ld_wait16(r);
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]) + lb;
                // (row of x: c0 + j)
                uint16_t *o = out + (size_t)(t.p0 + c0) * a.N + n;
                const int left = t.rows - c0;
                if constexpr (PARTIAL) {
                    float *s = a.sums + ((size_t)t.part * a.P + t.p0 + c0) * sum_pitch(a.N) + n;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n < a.N && j < left) s[(size_t)j * sum_pitch(a.N)] = v[j];
                } else if constexpr (MODE == kInner) {
                    uint16_t *h = out + n;
                    const int to = __ldg(a.rows + t.p0 + c0 + min(lane & 15, left - 1));
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int row = __shfl_sync(kAll, to, j);
                        if (n < a.N && j < left) {
                            uint32_t high, low;
                            two_bf16(f * v[j], high, low);
                            h[(size_t)row * 2 * a.N] = (uint16_t)high;
                            h[((size_t)row * 2 + 1) * a.N] = (uint16_t)low;
                        }
                    }
                } else if constexpr (SWIGLU) {
                    float f[8];  // row 2 i (gate lanes) or 2 i + 1 (up lanes) of output n
                    const bool up = lane >= 16;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float got = __shfl_xor_sync(kAll, up ? v[2 * i] : v[2 * i + 1], 16);
                        const float g = up ? got : v[2 * i], w = up ? v[2 * i + 1] : got;
                        f[i] = silu(g) * w;
                    }
                    o += up ? a.N : 0;
                    if (pairs) {  // two outputs a store: even lanes take f[i] of their neighbour's output too, odd ones f[i + 1]
                        const bool odd = lane & 1;
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float got = __shfl_xor_sync(kAll, odd ? f[i] : f[i + 1], 1);
                            const int j = 2 * i + (odd ? 2 : 0);
                            if (n < a.N && j + up < left)
                                *reinterpret_cast<uint32_t *>(o + (size_t)j * a.N - odd) =
                                    odd ? pack_bf16x2(got, f[i + 1]) : pack_bf16x2(f[i], got);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (n < a.N && 2 * i + up < left) o[(size_t)(2 * i) * a.N] = f32_to_bf16(f[i]);
                    }
                } else if (pairs) {
                    const bool odd = lane & 1;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float got = __shfl_xor_sync(kAll, odd ? v[j] : v[j + 1], 1);
                        if (n < a.N && j + odd < left)
                            *reinterpret_cast<uint32_t *>(o + (size_t)(j + odd) * a.N - odd) =
                                odd ? pack_bf16x2(got, v[j + 1]) : pack_bf16x2(v[j], got);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n < a.N && j < left) o[(size_t)j * a.N] = f32_to_bf16(v[j]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    mbar_arrive(&sh.acc_empty[b]);
                else
                    mbar_arrive_cluster(acc_empty0 + (uint32_t)(b * sizeof(uint64_t)));
            }
            if (!have) break;
        }
    }

    tc_fence_before();
    __syncthreads();
    // Drain TMA copies that were issued but never consumed (only after a timeout).
    if (tid == 0 && leader) {
        for (int i = sh.consumed; i < sh.issued; ++i)
            if (!mbar_wait(&sh.full[i % stages], (i / stages) & 1, status, kSiteDrain)) break;
    }
    // No remote arrival, copy or MMA operand read is left in flight past here.
    cluster_arrive_release();
    cluster_wait_acquire();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, tmem_cols);
    }
}

constexpr int kMaxDevices = 64;
int g_clusters[kMaxDevices];  // co-resident clusters of 2, per device

// The ring takes what shared memory there is, up to kMaxStages.
constexpr int kSmem = 232448;
int stages_of(int mode, int bt) {
    const int n = (kSmem - 1024 - (int)sizeof(GroupedShared)) / (kChunks * (w_bytes(mode) + bt * kChunkK));
    return n < kMaxStages ? n : kMaxStages;
}
int smem_of(int mode, int bt) {
    const int need = 1024 + stages_of(mode, bt) * kChunks * (w_bytes(mode) + bt * kChunkK) + (int)sizeof(GroupedShared);
    return need > 116 * 1024 ? need : 116 * 1024;  // one CTA per SM: the accumulators may be all of TMEM
}
static_assert(sizeof(GroupedShared) >= kWBytes / 2, "kInner's MMAs read past their rows, within shared memory");

using GroupedFn = void (*)(const CUtensorMap, const CUtensorMap, const RowMaps, const GroupedArgs, int, int, int, int,
                           int32_t *);

GroupedFn pick(int mode, bool gather, bool partial) {
    switch (mode) {
        case kInner: return grouped_kernel<kInner, true, false>;
        case kOuter: return partial ? grouped_kernel<kOuter, true, true> : grouped_kernel<kOuter, true, false>;
        case kSwiglu: return gather ? grouped_kernel<kSwiglu, true, false> : grouped_kernel<kSwiglu, false, false>;
        default:
            if (partial) return gather ? grouped_kernel<kPlain, true, true> : grouped_kernel<kPlain, false, true>;
            return gather ? grouped_kernel<kPlain, true, false> : grouped_kernel<kPlain, false, false>;
    }
}

// The parts of K added up, in order: out[p][n] (SwiGLU: of the sums' columns n and N + n), one output a thread.  The rows
// of no group, before the first and behind the last, stay as they are.
constexpr int kSumThreads = 256;
template <bool SWIGLU>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const float *__restrict__ sums, const int32_t *__restrict__ offsets,
                                                          int groups, int splits, int P, int N, uint16_t *__restrict__ out) {
    __shared__ int last;
    pdl_launch_dependents();
    pdl_wait();
    int first = 0, end = P;
    if (offsets) {
        if (threadIdx.x == 0) last = 0;
        __syncthreads();
        int most = 0;
        for (int e = threadIdx.x; e <= groups; e += kSumThreads) most = max(most, min(max(__ldg(offsets + e), 0), P));
        most = __reduce_max_sync(kAll, most);
        if ((threadIdx.x & 31) == 0) atomicMax(&last, most);
        __syncthreads();
        first = min(max(__ldg(offsets), 0), P);
        end = last;
    }
    const int pitch = sum_pitch(SWIGLU ? 2 * N : N);
    const size_t plane = (size_t)P * pitch;
    for (long long i = (long long)blockIdx.x * kSumThreads + threadIdx.x; i < (long long)P * N;
         i += (long long)gridDim.x * kSumThreads) {
        const int p = (int)(i / N), n = (int)(i - (long long)p * N);
        if (p < first || p >= end) continue;
        const float *s = sums + (size_t)p * pitch + n;
        float v = 0.0f, up = 0.0f;
#pragma unroll 8
        for (int k = 0; k < splits; ++k) {
            v += s[k * plane];
            if (SWIGLU) up += s[k * plane + N];
        }
        out[i] = f32_to_bf16(SWIGLU ? silu(v) * up : v);
    }
}

int launch_sum(bool swiglu, const float *sums, const int32_t *offsets, int groups, int splits, int P, int N, void *out,
               int num_sms, uint32_t flags, void *stream) {
    const long long blocks = ((long long)P * N + kSumThreads - 1) / kSumThreads, most = 8ll * num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(kSumThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, swiglu ? sum_kernel<true> : sum_kernel<false>, sums, offsets, groups, splits, P, N,
                                   static_cast<uint16_t *>(out));
}

cudaLaunchConfig_t config(int clusters, bool gather, int smem, uint32_t flags, void *stream, cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters));
    cfg.blockDim = dim3((unsigned)threads_of(gather));
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

// Co-resident clusters of 2 of the current device.
int clusters_of(int num_sms) {
    int dev = 0;
    const bool known = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices && g_clusters[dev] > 0;
    return known ? g_clusters[dev] : num_sms / 2;
}

// Tiles of up to bt rows and wt outputs; `full`: groups that may have rows.
int launch_mode(int mode, const GroupedArgs &a, int bt, int wt, int full, int num_sms, uint32_t flags, void *stream,
                int32_t *status, bool partial) {
    const bool swiglu = mode == kSwiglu;
    CUtensorMap tw, tb = {};
    RowMaps tx = {};
    // SwiGLU: blocks of 16 gate rows and their 16 up rows, all of a stage's in one box where no block runs past N
    const int w_boxes = swiglu && a.N % 16 ? 4 : 1;
    const uint64_t planes = mode == kOuter ? 1 : (uint64_t)a.groups, N = (uint64_t)a.N, K = (uint64_t)a.K;
    int r = swiglu && w_boxes == 1
                ? make_tmap_bf16_blocks(&tw, a.w, planes, 2, N, K, 16, 4, kChunkK)
                : make_tmap_bf16_stack(&tw, a.w, planes, swiglu ? 2 : 1, N, K, swiglu ? 2 : 1, swiglu ? 16 : (uint32_t)wt / 2,
                                       kChunkK);
    for (int i = mode == kOuter ? 3 : 0; i < 4 && !r && (!a.rows || mode == kOuter); ++i)
        r = make_tmap_bf16_2d(&tx.of[i], a.x, (uint64_t)a.x_rows, K, 16u << i, kChunkK, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (!r && mode == kOuter)
        r = make_tmap_bf16_stack(&tb, a.b, (uint64_t)a.groups, 1, N, (uint64_t)a.R, 1, (uint32_t)wt / 2, kRank);
    if (r) return (int)cudaErrorInvalidValue;
    // A cluster that cannot be resident with the others would run its tiles after them.
    const long long units = ((long long)a.P / bt + full) * ((a.N + wt - 1) / wt) *
                            (a.splits > 1 ? a.splits : 1);  // at most
    long long clusters = clusters_of(num_sms);
    if (units < clusters) clusters = units;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config((int)clusters, a.rows != nullptr, smem_of(mode, bt), flags, stream, attr);
    return (int)cudaLaunchKernelEx(&cfg, pick(mode, a.rows != nullptr, partial), tw, tb, tx, a, w_boxes, bt, wt,
                                   stages_of(mode, bt), status);
}

}  // namespace

int init_grouped() {
    for (int mode : {kPlain, kSwiglu, kInner, kOuter})
        for (bool gather : {false, true})
            for (bool partial : {false, true}) {
                const int e = (int)cudaFuncSetAttribute(pick(mode, gather, partial),
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
                if (e) return e;
            }
    int dev = 0;
    const int e = (int)cudaGetDevice(&dev);
    if (e || dev < 0 || dev >= kMaxDevices) return e ? e : (int)cudaErrorInvalidDevice;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(kGb300Sms, true, kSmem, 0, nullptr, attr);
    cfg.numAttrs = 1;
    int n = 0;
    // A failed query only loses the clamp (launches then use half the SMs' number).
    if (cudaOccupancyMaxActiveClusters(&n, pick(kPlain, true, false), &cfg) != cudaSuccess) {
        n = 0;
        (void)cudaGetLastError();
    }
    g_clusters[dev] = n;
    return 0;
}

namespace {

// Rows of a tile: groups of the average size, and of twice that, fit one.
int tile_rows(int P, int groups) {
    const long long twice = 2ll * P / (P < groups ? P : groups);
    return twice <= 32 ? 32 : twice <= 64 ? 64 : twice <= 128 ? 128 : 256;
}

// Parts of K for `units` tiles: where they leave half of the pairs of SMs without one, as many parts as there are pairs for,
// at most eight, of four stages at least.
int parts_of(long long units, int K) {
    constexpr int pairs = kGb300Sms / 2;
    if (2 * units > pairs) return 1;
    const long long stages = K / (kChunkK * kChunks) / 4, s = pairs / units < stages ? pairs / units : stages;
    return s < 2 ? 1 : s < 8 ? (int)s : 8;
}

}  // namespace

// (a group of P rows may be one tile more than its share; SwiGLU's wide product is summed as it is)
int grouped_splits(int P, int groups, int N, int K, int swiglu) {
    if (P <= 0) return 1;
    const long long tiles = (long long)P / tile_rows(P, groups) + (P < groups ? P : groups);
    return parts_of(tiles * (((swiglu ? 2ll : 1ll) * N + 255) / 256), K);
}
int lora_outer_splits(int M, int N, int K) {
    return parts_of(((long long)M + 255) / 256 * (((long long)N + 127) / 128), K);
}

int launch_grouped(const GroupedArgs &a, int num_sms, uint32_t flags, void *stream, int32_t *status) {
    const int full = a.P < a.groups ? a.P : a.groups, bt = tile_rows(a.P, a.groups);
    if (a.splits > 1) {
        GroupedArgs p = a;
        p.N = a.swiglu ? 2 * a.N : a.N;
        const int r = launch_mode(kPlain, p, bt, 256, full, num_sms, flags, stream, status, true);
        if (r) return r;
        return launch_sum(a.swiglu != 0, a.sums, a.offsets, a.groups, a.splits, a.P, a.N, a.out, num_sms, flags, stream);
    }
    return launch_mode(a.swiglu ? kSwiglu : kPlain, a, bt, a.swiglu ? 128 : 256, full, num_sms, flags, stream, status, false);
}

// (the rows' number is known here: tiles of no more)
int lora_base_splits(int M, int N, int K) {
    const int bt = M <= 128 ? 128 : 256;
    return parts_of(((long long)M + bt - 1) / bt * (((long long)N + 255) / 256), K);
}
int launch_lora_base(const LoraArgs &l, const void *w, const void *bias, int num_sms, uint32_t flags, void *stream,
                     int32_t *status) {
    const GroupedArgs a = {l.x, w, bias, l.span, nullptr, nullptr, l.M, l.M, 1, l.N, l.K, 0, nullptr, nullptr, nullptr, 0,
                           l.sums, l.parts};
    return launch_mode(kPlain, a, l.M <= 128 ? 128 : 256, 256, 1, num_sms, flags, stream, status, true);
}

int launch_lora_inner_grouped(const LoraArgs &l, const int32_t *offsets, const int32_t *rows, int num_sms, uint32_t flags,
                              void *stream, int32_t *status) {
    const GroupedArgs a = {l.x, l.a, nullptr, offsets, rows, l.h, l.M, l.M, l.L, l.R, l.K, 0, l.scale, nullptr, nullptr, 0,
                           nullptr, 1};
    // One W tile, half of its rows each CTA's: rows of x so that there is a tile for each pair of SMs.
    const int clusters = clusters_of(num_sms);
    const int bt = l.M <= 32 * clusters ? 32 : l.M <= 64 * clusters ? 64 : l.M <= 128 * clusters ? 128 : 256;
    return launch_mode(kInner, a, bt, (l.R + 15) / 16 * 16, l.M < l.L ? l.M : l.L, num_sms, flags, stream, status, false);
}

int launch_lora_outer_grouped(const LoraArgs &l, const void *w, const void *bias, const int32_t *offsets, const int32_t *rows,
                              int num_sms, uint32_t flags, void *stream, int32_t *status) {
    const GroupedArgs a = {l.x, w, bias, offsets, rows, l.out, l.M, l.M, l.L, l.N, l.K, 0, nullptr, l.b, l.h, l.R,
                           l.sums, lora_outer_splits(l.M, l.N, l.K)};
    if (a.splits > 1) {
        const int r = launch_mode(kOuter, a, 256, 128, 1, num_sms, flags, stream, status, true);
        if (r) return r;
        return launch_sum(false, a.sums, nullptr, 0, a.splits, a.P, a.N, a.out, num_sms, flags, stream);
    }
    // The width that needs the least time, a round of tiles going with its width and a share for x (256 x 14336 x 4096: 75
    // tiles of 192 on 76 pairs, 56 of 256).
    const int clusters = clusters_of(num_sms);
    int wt = 256;
    long long best = 0;
    for (int w0 = 256; w0 >= 128; w0 -= 32) {
        const long long units = (((long long)l.M + 255) / 256) * ((l.N + w0 - 1) / w0);
        const long long cost = (units + clusters - 1) / clusters * (w0 + 64);
        if (best == 0 || cost < best) {
            best = cost;
            wt = w0;
        }
    }
    return launch_mode(kOuter, a, 256, wt, 1, num_sms, flags, stream, status, false);
}

}  // namespace bf16l
