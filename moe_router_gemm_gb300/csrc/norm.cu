// norm.cu — root-mean-square norm of rows, with the residual's addition before
// it and an output in bf16 and / or in 8 or 4 bits with scales.
//
//     h = x  or  RNE_bf16(x + residual);  y = h / sqrt(mean(h^2) + eps) * weight
//
// One pass: a row stays on the SM between the sum of squares and the output, so each
// input is read from memory once and each output written once: HBM is the bound.  The sum
// runs in fp32: each thread over its own values in order, then a butterfly, then the
// warps' sums by a butterfly, so it is the same from run to run.
//
//   * norm_vec_kernel: rows that start on 16-byte boundaries (H and ldx multiples of
//     8): a row to a warp (H <= 1024) or to a block; thread i holds the 8-value vectors
//     i, i + threads, ...; four neighbouring lanes hold a 32-element scale block.  The
//     weight stays in registers from row to row, and the next row's loads go out
//     before this row's sum, so memory is busy through the reduction.  8192 x 7168
//     with a residual: 71 us to bf16 (97% of the copy bandwidth), 83 us to bf16 and
//     MXFP8 (94%); without one 40.4 us (86%), and 59 to bf16 and MXFP8 (74%) or MXFP4
//     (66%).  Not all of a row is in registers everywhere: blocks of up to 1024 threads
//     have 64 a thread, of which two vectors with MX output spill 32 to 36 bytes, and four
//     (H above 16384) 188 to 288: 8192 x 20000 212 us (45%).
//   * norm_shift_kernel: odd lengths and strides.  The dense tensors' vectors start on
//     16-byte boundaries, so a row is up to 7 values, vectors, up to 7 values; a
//     vector of x that lies across two 16-byte blocks is shifted out of both; the
//     weight, which meets the vectors at a different place in every row, comes from
//     shared memory.  A value at a time these took 1.5 to 3 times as long: 2000 x 2881
//     with a residual 27 us (10.2 here; floor 6.8), 8192 x 7168 of 7300 columns 114 (78;
//     34.6), 8192 x 7168 of 7169 columns with MXFP8 295 (100; 43.5).  8192 x 5001 of 5200
//     takes 71 (24.1).  So 29 to 67% of the floor's rate is reached and HBM is not the
//     bound; the weight comes in 4-byte reads, four lanes to a bank, even where H % 8 == 0
//     and registers could keep it, and two shifted vectors a thread spill 36 to 204 bytes.
//     (The second block from the next lane instead of a load of its own: 2048 x 1536 of
//     2113 columns 11.5 us, 6.3 with the load.)
//   * norm_any_kernel: what is left (off 16-byte boundaries: H below 64 or above 16384; on
//     them: H above 32768): one value per lane and step; a warp's 32 lanes hold a scale
//     block.  Long rows are read twice (the second time from L1 or L2).
#include <cuda_runtime.h>

#include "moe.h"
#include "mxfp4.cuh"

namespace bf16l {

namespace {

struct NormArgs {
    const uint16_t *x;
    const uint16_t *residual;
    const uint16_t *weight;
    uint16_t *out;
    uint16_t *residual_out;
    uint8_t *codes;
    uint8_t *scales;
    const float *scale;
    long long rows, ldx;
    int H;
    float eps;
};

__device__ __forceinline__ uint16_t e4m3x2_sat(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the block, the same in every thread.  `red`: 32 floats, alternating between two buffers from call to call
// (one barrier a call: whoever writes a buffer again has passed the barrier after its last readers).
__device__ __forceinline__ float block_sum(float v, float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (int)blockDim.x >> 5;
    v = warp_sum(v);
    if (nw == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < nw ? red[lane] : 0.0f);
}

// Magnitude bits of a value for a block's maximum: NaN above infinity, so it shows.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The outputs of eight values from element `at` of the dense tensors on (a multiple of 8).  For the MX formats the
// four lanes of a quad hold a block and call it together.
template <int QUANT>
__device__ __forceinline__ void put8(const NormArgs &a, long long at, float (&y)[8], float inv_scale) {
    if (a.out) OutStore<uint16_t>::eight(a.out + at, y);
    if (QUANT == BF16L_QUANT_NONE) return;
    float f = inv_scale;
    bool nan = false;
    if (QUANT != BF16L_QUANT_FP8) {
        const unsigned quad = 0xFu << (threadIdx.x & 28u);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, mag_bits(y[e]));
        m = max(m, __shfl_xor_sync(quad, m, 1));
        m = max(m, __shfl_xor_sync(quad, m, 2));
        nan = m > 0x7F800000u;
        const int s = mx_scale_exp(m, QUANT == BF16L_QUANT_MXFP8 ? 8 : 2);
        f = exp2_neg(nan ? 0 : s);
        if ((threadIdx.x & 3) == 0) a.scales[at >> 5] = nan ? 255 : (uint8_t)(s + 127);
    }
    if (QUANT == BF16L_QUANT_MXFP4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= f;
        *reinterpret_cast<uint32_t *>(a.codes + (at >> 1)) = nan ? 0u : e2m1x8(y);
    } else {
        uint16_t d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = e4m3x2_sat(y[2 * e] * f, y[2 * e + 1] * f);
        *reinterpret_cast<uint2 *>(a.codes + at) =
            make_uint2((uint32_t)d[0] | ((uint32_t)d[1] << 16), (uint32_t)d[2] | ((uint32_t)d[3] << 16));
    }
}

__device__ __forceinline__ uint4 add_bf16x8(const uint4 &h, const uint4 &q) {
    return make_uint4(pack_bf16x2(bf16_lo(h.x) + bf16_lo(q.x), bf16_hi(h.x) + bf16_hi(q.x)),
                      pack_bf16x2(bf16_lo(h.y) + bf16_lo(q.y), bf16_hi(h.y) + bf16_hi(q.y)),
                      pack_bf16x2(bf16_lo(h.z) + bf16_lo(q.z), bf16_hi(h.z) + bf16_hi(q.z)),
                      pack_bf16x2(bf16_lo(h.w) + bf16_lo(q.w), bf16_hi(h.w) + bf16_hi(q.w)));
}

__device__ __forceinline__ float squares(const uint4 &v, float ss) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ss = fmaf(bf16_lo(u[e]), bf16_lo(u[e]), ss);
        ss = fmaf(bf16_hi(u[e]), bf16_hi(u[e]), ss);
    }
    return ss;
}

__device__ __forceinline__ void scaled(float (&y)[8], const uint4 &v, float rstd, const uint4 &w) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w}, g[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        y[2 * e] = bf16_lo(u[e]) * rstd * bf16_lo(g[e]);
        y[2 * e + 1] = bf16_hi(u[e]) * rstd * bf16_hi(g[e]);
    }
}

// V: vectors per thread.  WARP: a row to a warp, else to a block.  T: at most this many threads.
template <int QUANT, int V, bool WARP, int T>
__global__ void __launch_bounds__(T) norm_vec_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();  // x, the residual, the weight and the scale may be written by the previous kernel
    const int nvec = a.H >> 3, nt = WARP ? 32 : (int)blockDim.x, me = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long step = WARP ? (long long)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    long long r = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const float inv_scale = QUANT == BF16L_QUANT_FP8 ? 1.0f / __ldg(a.scale) : 0.0f;
    const uint4 kNone = make_uint4(0u, 0u, 0u, 0u);
    uint4 w[V], h[V], q[V];
    auto load = [&](long long row) {
        const uint4 *xr = reinterpret_cast<const uint4 *>(a.x + row * a.ldx);
        const uint4 *rr = reinterpret_cast<const uint4 *>(a.residual + row * a.H);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            h[j] = i < nvec ? __ldg(xr + i) : kNone;
            if (a.residual) q[j] = i < nvec ? rr[i] : kNone;  // (may be written in place: not __ldg)
        }
    };
    if (r < a.rows) load(r);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = me + j * nt;
        w[j] = i < nvec ? __ldg(reinterpret_cast<const uint4 *>(a.weight) + i) : kNone;
    }
    for (int par = 0; r < a.rows; r += step, par ^= 1) {
        uint4 c[V];  // this row's h
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] = a.residual ? add_bf16x8(h[j], q[j]) : h[j];
        if (r + step < a.rows) load(r + step);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            if (a.residual && i < nvec) reinterpret_cast<uint4 *>(a.residual_out + r * a.H)[i] = c[j];
            ss = squares(c[j], ss);
        }
        const float rstd = 1.0f / sqrtf((WARP ? warp_sum(ss) : block_sum(ss, red[par])) / (float)a.H + a.eps);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            if (i >= nvec) break;  // nvec % 4 == 0 for the MX formats: a quad leaves together
            float y[8];
            scaled(y, c[j], rstd, w[j]);
            put8<QUANT>(a, r * a.H + 8 * (long long)i, y, inv_scale);
        }
    }
}

// Eight bf16 weights from element i on (any i), from a copy in shared memory that is two words longer than the weight.
__device__ __forceinline__ uint4 weights_at(const uint32_t *w, int i) {
    const uint32_t *p = w + (i >> 1);
    if ((i & 1) == 0) return make_uint4(p[0], p[1], p[2], p[3]);
    return make_uint4(__funnelshift_r(p[0], p[1], 16), __funnelshift_r(p[1], p[2], 16), __funnelshift_r(p[2], p[3], 16),
                      __funnelshift_r(p[3], p[4], 16));
}

// The 16-byte block at p (16-byte aligned), of which only the part inside [lo, hi) is read.
__device__ __forceinline__ uint4 load_block(const uint16_t *p, const uint16_t *lo, const uint16_t *hi) {
    if (p >= lo && p + 8 <= hi) return __ldg(reinterpret_cast<const uint4 *>(p));
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < 8; ++i)
        if (p + i >= lo && p + i < hi) w[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sixteen bytes from byte m (even, below 16) of two neighbouring blocks on (shift_blocks, less the odd places).
__device__ __forceinline__ uint4 shift_blocks_even(const uint4 &a, const uint4 &b, int m) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t v[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {  // words m / 4 + k
        const uint32_t lo = m & 4 ? w[k + 1] : w[k], hi = m & 4 ? w[k + 3 < 8 ? k + 3 : 7] : w[k + 2];
        v[k] = m & 8 ? hi : lo;
    }
    if ((m & 2) == 0) return make_uint4(v[0], v[1], v[2], v[3]);
    return make_uint4(__funnelshift_r(v[0], v[1], 16), __funnelshift_r(v[1], v[2], 16), __funnelshift_r(v[2], v[3], 16),
                      __funnelshift_r(v[3], v[4], 16));
}

// V: vectors per thread.  XS: the vectors of x are not all on 16-byte boundaries.
template <int QUANT, int V, bool XS>
__global__ void __launch_bounds__(1024) norm_shift_kernel(const NormArgs a) {
    extern __shared__ uint32_t sw[];  // the weight
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int nt = (int)blockDim.x, me = (int)threadIdx.x;
    const float inv_scale = QUANT == BF16L_QUANT_FP8 ? 1.0f / __ldg(a.scale) : 0.0f;
    const uint4 kNone = make_uint4(0u, 0u, 0u, 0u);
    const uint16_t *xend = a.x + (a.rows - 1) * a.ldx + a.H;
    uint4 h[V], h2[XS ? V : 1], q[V];
    uint16_t hs = 0, qs = 0;     // threads 0-7: the values before the first vector; 8-15: those after the last
    int head, nv, edge, xm = 0;  // of the row that is loaded; edge: this thread's single value, or -1
    auto load = [&](long long row) {
        head = (int)(-(row * a.H) & 7);
        if (head > a.H) head = a.H;
        nv = (a.H - head) >> 3;
        const int end = head + 8 * nv;
        edge = me < head ? me : me >= 8 && me < 16 && end + me - 8 < a.H ? end + me - 8 : -1;
        const uint16_t *x = a.x + row * a.ldx, *r = a.residual + row * a.H;
        if (edge >= 0) {
            hs = x[edge];
            if (a.residual) qs = r[edge];
        }
        if (XS) xm = (int)(reinterpret_cast<uintptr_t>(x + head) & 15u);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            if (XS) {
                const uint16_t *b = x + head + 8 * i - (xm >> 1);
                h[j] = i < nv ? load_block(b, a.x, xend) : kNone;
                h2[j] = i < nv && xm ? load_block(b + 8, a.x, xend) : kNone;
            } else {
                h[j] = i < nv ? __ldg(reinterpret_cast<const uint4 *>(x + head) + i) : kNone;
            }
            if (a.residual) q[j] = i < nv ? reinterpret_cast<const uint4 *>(r + head)[i] : kNone;
        }
    };
    long long r = blockIdx.x;
    if (r < a.rows) load(r);
    for (int i = me; i < (a.H + 1) / 2 + 2; i += nt) {
        const uint32_t lo = 2 * i < a.H ? __ldg(a.weight + 2 * i) : 0u;
        const uint32_t hi = 2 * i + 1 < a.H ? __ldg(a.weight + 2 * i + 1) : 0u;
        sw[i] = lo | hi << 16;
    }
    __syncthreads();
    for (int par = 0; r < a.rows; r += gridDim.x, par ^= 1) {
        uint4 c[V];
        float ss = 0.0f, cs = 0.0f;
        const int chead = head, cnv = nv, cedge = edge;
        const long long at = r * a.H;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            c[j] = XS ? shift_blocks_even(h[j], h2[XS ? j : 0], xm) : h[j];
            if (a.residual) c[j] = add_bf16x8(c[j], q[j]);
        }
        if (cedge >= 0) {
            uint16_t b = hs;
            if (a.residual) {
                b = f32_to_bf16(bf16_to_f32(hs) + bf16_to_f32(qs));
                a.residual_out[at + cedge] = b;
            }
            cs = bf16_to_f32(b);
            ss = cs * cs;
        }
        if (r + gridDim.x < a.rows) load(r + gridDim.x);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            if (i >= cnv) break;  // (what lies there of x is not this row's)
            if (a.residual) reinterpret_cast<uint4 *>(a.residual_out + at + chead)[i] = c[j];
            ss = squares(c[j], ss);
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red[par]) / (float)a.H + a.eps);
        if (cedge >= 0) {  // (never for the MX formats: their rows are whole vectors)
            const uint32_t w = sw[cedge >> 1];
            const float y = cs * rstd * (cedge & 1 ? bf16_hi(w) : bf16_lo(w));
            if (a.out) a.out[at + cedge] = f32_to_bf16(y);
            if (QUANT == BF16L_QUANT_FP8) a.codes[at + cedge] = (uint8_t)(e4m3x2_sat(y * inv_scale, 0.0f) & 0xFFu);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = me + j * nt;
            if (i >= cnv) break;  // a quad leaves together, as in norm_vec_kernel
            float y[8];
            scaled(y, c[j], rstd, weights_at(sw, chead + 8 * i));
            put8<QUANT>(a, at + chead + 8 * (long long)i, y, inv_scale);
        }
    }
}

// N: values per thread that stay in registers (0: the row is read again).
template <int QUANT, int N>
__global__ void __launch_bounds__(1024) norm_any_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int nt = (int)blockDim.x, lane = threadIdx.x & 31;
    const float inv_scale = QUANT == BF16L_QUANT_FP8 ? 1.0f / __ldg(a.scale) : 0.0f;
    int par = 0;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x, par ^= 1) {
        const uint16_t *xr = a.x + r * a.ldx;
        const uint16_t *hr = a.residual ? a.residual_out + r * a.H : xr;  // where h is read from the second time
        float h[N ? N : 1], ss = 0.0f;
        auto add = [&](uint16_t xv, uint16_t qv, int i) {
            float v = bf16_to_f32(xv);
            if (a.residual) {
                const uint16_t b = f32_to_bf16(v + bf16_to_f32(qv));
                a.residual_out[r * a.H + i] = b;
                v = bf16_to_f32(b);
            }
            return v;
        };
        if constexpr (N > 0) {
            uint16_t xv[N], qv[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = (int)threadIdx.x + j * nt;
                xv[j] = i < a.H ? xr[i] : (uint16_t)0;
                qv[j] = a.residual && i < a.H ? a.residual[r * a.H + i] : (uint16_t)0;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = (int)threadIdx.x + j * nt;
                h[j] = i < a.H ? add(xv[j], qv[j], i) : 0.0f;
                ss = fmaf(h[j], h[j], ss);
            }
        } else {
            for (unsigned i = threadIdx.x; i < (unsigned)a.H; i += nt) {  // (H may be within a block of 2^31)
                const float v = add(xr[i], a.residual ? a.residual[r * a.H + i] : (uint16_t)0, (int)i);
                ss = fmaf(v, v, ss);
            }
        }
        const float rstd = 1.0f / sqrtf(block_sum(ss, red[par]) / (float)a.H + a.eps);
        auto put = [&](float v, int i) {
            const float y = v * rstd * bf16_to_f32(__ldg(a.weight + i));
            if (a.out) a.out[r * a.H + i] = f32_to_bf16(y);
            if (QUANT == BF16L_QUANT_FP8) {
                a.codes[r * a.H + i] = (uint8_t)(e4m3x2_sat(y * inv_scale, 0.0f) & 0xFFu);
            } else if (QUANT != BF16L_QUANT_NONE) {  // H % 32 == 0: a warp's lanes are one block, together here
                uint32_t m = mag_bits(y);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const bool nan = m > 0x7F800000u;
                const int s = mx_scale_exp(m, QUANT == BF16L_QUANT_MXFP8 ? 8 : 2);
                const float t = y * exp2_neg(nan ? 0 : s);
                if (QUANT == BF16L_QUANT_MXFP8) {
                    a.codes[r * a.H + i] = (uint8_t)(e4m3x2_sat(t, 0.0f) & 0xFFu);
                } else {
                    const float w[8] = {t, __shfl_down_sync(0xFFFFFFFFu, t, 1), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    const uint32_t c = nan ? 0u : e2m1x8(w);
                    if ((lane & 1) == 0) a.codes[r * (a.H >> 1) + (i >> 1)] = (uint8_t)c;
                }
                if (lane == 0) a.scales[r * (a.H >> 5) + (i >> 5)] = nan ? 255 : (uint8_t)(s + 127);
            }
        };
        if constexpr (N > 0) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int i = (int)threadIdx.x + j * nt;
                if (i < a.H) put(h[j], i);
            }
        } else {
            // (h was written by this same thread)
            for (unsigned i = threadIdx.x; i < (unsigned)a.H; i += nt) put(bf16_to_f32(hr[i]), (int)i);
        }
    }
}

using NormFn = void (*)(const NormArgs);

template <int QUANT>
NormFn pick_vec(int v, bool warp, int threads) {
    if (warp)
        return v == 1   ? norm_vec_kernel<QUANT, 1, true, 256>
               : v == 2 ? norm_vec_kernel<QUANT, 2, true, 256>
                        : norm_vec_kernel<QUANT, 4, true, 256>;
    if (v == 4) return threads <= 512 ? norm_vec_kernel<QUANT, 4, false, 512> : norm_vec_kernel<QUANT, 4, false, 1024>;
    return v == 1 ? norm_vec_kernel<QUANT, 1, false, 1024> : norm_vec_kernel<QUANT, 2, false, 1024>;
}

template <int QUANT>
NormFn pick_shift(int v, bool xs) {
    if (xs) return v == 1 ? norm_shift_kernel<QUANT, 1, true> : norm_shift_kernel<QUANT, 2, true>;
    return v == 1 ? norm_shift_kernel<QUANT, 1, false> : norm_shift_kernel<QUANT, 2, false>;
}

template <int QUANT>
NormFn pick_any(int n) {
    return n == 4 ? norm_any_kernel<QUANT, 4> : norm_any_kernel<QUANT, 0>;
}

}  // namespace

int launch_rmsnorm(const void *x, int64_t ldx, const void *residual, const void *weight, void *out, void *residual_out,
                   void *codes, void *scales, const float *scale, int64_t rows, int H, float eps, int quant,
                   int num_sms, uint32_t flags, void *stream) {
    NormArgs a = {static_cast<const uint16_t *>(x),
                  static_cast<const uint16_t *>(residual),
                  static_cast<const uint16_t *>(weight),
                  static_cast<uint16_t *>(out),
                  static_cast<uint16_t *>(residual_out),
                  static_cast<uint8_t *>(codes),
                  static_cast<uint8_t *>(scales),
                  scale,
                  rows,
                  ldx,
                  H,
                  eps};
    const bool vec = H % 8 == 0 && ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && H <= 8 * 4 * 1024;
    int threads;
    long long blocks;
    size_t smem = 0;
    NormFn fn;
    if (vec) {
        const int nvec = H / 8;
        const bool warp = nvec <= 128;
        // Long rows with a residual: four vectors a thread (8192 x 7168 with MXFP8 83 us, 91 with two; 8192 x 4096 with
        // MXFP4 44.7 and 46.3 with one).  Without one, or short, fewer: 8192 x 7168 40.5 us with two, 43 with four;
        // 2048 x 2880 with a residual 7.8 and 9.
        const int v = warp ? (nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4)
                      : residual && nvec >= 512 ? 4 : nvec <= 512 ? 1 : nvec <= 2048 ? 2 : 4;
        threads = warp ? 256 : ((nvec + v - 1) / v + 31) / 32 * 32;
        blocks = warp ? (rows + 7) / 8 : rows;
        fn = quant == BF16L_QUANT_NONE    ? pick_vec<BF16L_QUANT_NONE>(v, warp, threads)
             : quant == BF16L_QUANT_FP8   ? pick_vec<BF16L_QUANT_FP8>(v, warp, threads)
             : quant == BF16L_QUANT_MXFP8 ? pick_vec<BF16L_QUANT_MXFP8>(v, warp, threads)
                                           : pick_vec<BF16L_QUANT_MXFP4>(v, warp, threads);
    } else if (H >= 64 && H <= 16384) {
        const bool xs = (ldx - H) % 8 != 0 || (reinterpret_cast<uintptr_t>(x) & 15u) != 0;
        const int nvec = (H + 7) / 8, v = nvec <= (xs ? 1024 : 256) ? 1 : 2;
        threads = ((nvec + v - 1) / v + 31) / 32 * 32;
        blocks = rows;
        smem = ((size_t)(H + 1) / 2 + 2) * 4;
        fn = quant == BF16L_QUANT_NONE    ? pick_shift<BF16L_QUANT_NONE>(v, xs)
             : quant == BF16L_QUANT_FP8   ? pick_shift<BF16L_QUANT_FP8>(v, xs)
             : quant == BF16L_QUANT_MXFP8 ? pick_shift<BF16L_QUANT_MXFP8>(v, xs)
                                          : pick_shift<BF16L_QUANT_MXFP4>(v, xs);
    } else {
        const int n = H <= 64 ? 4 : 0;
        threads = n ? 32 : 512;
        blocks = rows;
        fn = quant == BF16L_QUANT_NONE    ? pick_any<BF16L_QUANT_NONE>(n)
             : quant == BF16L_QUANT_FP8   ? pick_any<BF16L_QUANT_FP8>(n)
             : quant == BF16L_QUANT_MXFP8 ? pick_any<BF16L_QUANT_MXFP8>(n)
                                           : pick_any<BF16L_QUANT_MXFP4>(n);
    }
    const long long cap = (long long)num_sms * (2048 / threads);
    if (blocks > cap) blocks = cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_attr_of(flags);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace bf16l
