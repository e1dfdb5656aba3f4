// sbl_ckpt.cuh -- the gated activation and the RMSNorm with 8-bit activation
// checkpoints (the b8 format) on sm_100a.
//
// Between two linears a training step keeps what their backward reads: the
// pre-activations of the MLP and the norms' inputs, 2 bytes an element.  The
// forward kernels here write them as b8 matrices instead (1 byte and 1/128),
// from the registers that hold the bf16 inputs anyway, and the backward
// kernels read only those.  The backward is the exact gradient of the formula
// at the checkpointed values.
#pragma once

#include "sbl_b8.cuh"

namespace sbl {

enum ActKind : int { kActSilu = 0, kActRelu2 = 1 };

// act(g), and act'(g) beside it.  relu2(g) = max(g, 0)^2, relu2' = 2 max(g, 0).
// silu(g) = g s, s = 1 / (1 + e^-g), silu' = s (1 + g (1 - s)), with
// t = e^-|g| <= 1:  s = (g < 0 ? t : 1) / (1 + t),  1 - s = (g < 0 ? 1 : t) / (1 + t),
// so that nothing overflows and far negative g keep their (tiny) values: t is
// the square of e^-|g|/2, which the flushing form of ex2 still holds.  t is off
// by about |g| 2^-23 and the reciprocal by 2^-23, far below the bf16 results'
// half step of 2^-8.
__device__ __forceinline__ float exp_neg_abs(float g)
{
    float h;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(__fmul_rn(fabsf(g), -0.72134752f)));  // -log2(e) / 2
    return __fmul_rn(h, h);
}

__device__ __forceinline__ float rcp_approx(float x)  // x in [1, 2]
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int ACT>
__device__ __forceinline__ float act_value(float g)
{
    if constexpr (ACT == kActRelu2) {
        const float p = g < 0.0f ? 0.0f : g;  // a NaN stays one
        return p * p;
    } else {
        const float t = exp_neg_abs(g);
        return g * ((g < 0.0f ? t : 1.0f) * rcp_approx(1.0f + t));
    }
}

template <int ACT>
__device__ __forceinline__ void act_value_grad(float g, float &a, float &da)
{
    if constexpr (ACT == kActRelu2) {
        const float p = g < 0.0f ? 0.0f : g;
        a = p * p;
        da = p + p;
    } else {
        const float t = exp_neg_abs(g), inv = rcp_approx(1.0f + t), ti = t * inv;
        const float s = g < 0.0f ? ti : inv, rest = g < 0.0f ? inv : ti;
        a = g * s;
        da = s * fmaf(g, rest, 1.0f);
    }
}

// h = act(g) u (u absent: h = act(g)), with the checkpoints of g and u.  The
// layout of the row quantiser: a warp per (row, 512 columns).  Memory bound:
// per element 4 bytes read, 2 + 2 written.
struct GluFwdArgs {
    const uint16_t *G, *U;  // U nullptr: not gated
    int64_t ldg, ldu;
    uint16_t *H;            // nullptr: only the checkpoints
    int64_t ldh;
    uint8_t *gc, *uc;       // checkpoint codes (nullptr: none)
    uint32_t *gs, *us;
    int64_t ldc;
    int64_t rp;
    int32_t rows, cols, words, per_warp, v32;
};

template <int TYPE, int ACT, bool GATED>
__global__ void __launch_bounds__(256) glu_forward_kernel(GluFwdArgs a)
{
    grid_wait_and_release();
    const int lane = threadIdx.x & 31;
    const B8Walk wk = b8_walk(a.words, a.per_warp);
    if (wk.row >= a.rp) return;
    const int64_t wi = b8_word_index(0, a.rp, wk.row);
    if (wk.row >= a.rows) {
        if (lane == 0)
            for (int w = wk.w0; w < wk.w1; w += wk.step) {
                if (a.gc) a.gs[wi + w * a.rp] = kB8PadWord;
                if (GATED && a.uc) a.us[wi + w * a.rp] = kB8PadWord;
            }
        return;
    }
    const uint16_t *G = a.G + wk.row * a.ldg, *U = GATED ? a.U + wk.row * a.ldu : nullptr;
    for (int w = wk.w0; w < wk.w1; w += wk.step) {
        const int c = 512 * w + 16 * lane;
        const bool ok = c < a.cols;
        Bf16x16 g = {}, u = {};
        if (ok) {
            g = load_bf16x16(G + c, a.v32);
            if (GATED) u = load_bf16x16(U + c, a.v32);
        }
        if (a.H && ok) {
            Bf16x16 h;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float lo = act_value<ACT>(bf16_lo(g.w[i])), hi = act_value<ACT>(bf16_hi(g.w[i]));
                if (GATED) lo *= bf16_lo(u.w[i]), hi *= bf16_hi(u.w[i]);
                h.w[i] = pack_bf16(lo, hi);
            }
            store_bf16x16(a.H + wk.row * a.ldh + c, h, a.v32);
        }
        // the largest magnitudes of both blocks in one reduction
        const uint32_t top = eighth_max2(bf16x16_absmax(g) | (GATED ? bf16x16_absmax(u) << 16 : 0u));
        if (a.gc) {
            const uint32_t byte = b8_scale_byte<TYPE>(top << 16);
            if (ok) *reinterpret_cast<uint4 *>(a.gc + wk.row * a.ldc + c) = b8_encode_bf16x16<TYPE>(g, b8_inv_scale(byte));
            const uint32_t word = scale_word(byte, lane);
            if (lane == 0) a.gs[wi + w * a.rp] = word;
        }
        if (GATED && a.uc) {
            const uint32_t byte = b8_scale_byte<TYPE>(top & 0xffff0000u);
            if (ok) *reinterpret_cast<uint4 *>(a.uc + wk.row * a.ldc + c) = b8_encode_bf16x16<TYPE>(u, b8_inv_scale(byte));
            const uint32_t word = scale_word(byte, lane);
            if (lane == 0) a.us[wi + w * a.rp] = word;
        }
    }
}

// dg = dh u act'(g), du = dh act(g) at the checkpointed g and u.
struct GluBwdArgs {
    const uint8_t *gc, *uc;
    const uint32_t *gs, *us;
    int64_t ldc, rp;
    const uint16_t *dH;
    int64_t ldh;
    uint16_t *dG, *dU;
    int64_t ldg, ldu;
    int32_t rows, cols, words, per_warp, v32;
};

template <int TYPE, int ACT, bool GATED>
__global__ void __launch_bounds__(256) glu_backward_kernel(GluBwdArgs a)
{
    grid_wait_and_release();
    const int lane = threadIdx.x & 31;
    const B8Walk wk = b8_walk(a.words, a.per_warp);
    if (wk.row >= a.rows) return;
    const int64_t wi = b8_word_index(0, a.rp, wk.row);
    for (int w = wk.w0; w < wk.w1; w += wk.step) {
        const int c = 512 * w + 16 * lane, sh = 8 * (lane >> 3);
        if (c >= a.cols) continue;
        const uint32_t gw = __ldg(a.gs + wi + w * a.rp), uw = GATED ? __ldg(a.us + wi + w * a.rp) : 0u;
        const uint4 gq = __ldg(reinterpret_cast<const uint4 *>(a.gc + wk.row * a.ldc + c));
        const uint4 uq = GATED ? __ldg(reinterpret_cast<const uint4 *>(a.uc + wk.row * a.ldc + c)) : make_uint4(0u, 0u, 0u, 0u);
        const Bf16x16 dh = load_bf16x16(a.dH + wk.row * a.ldh + c, a.v32);
        const float gsc = b8_scale((gw >> sh) & 0xffu), usc = GATED ? b8_scale((uw >> sh) & 0xffu) : 0.0f;
        const uint32_t gqw[4] = {gq.x, gq.y, gq.z, gq.w}, uqw[4] = {uq.x, uq.y, uq.z, uq.w};
        Bf16x16 dg, du;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float g[4], u[4], x[4], y[4];
            b8_decode4<TYPE>(gqw[i], g);
            if (GATED) b8_decode4<TYPE>(uqw[i], u);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t hw = dh.w[2 * i + (k >> 1)];
                const float d = k & 1 ? bf16_hi(hw) : bf16_lo(hw);
                float v, dv;
                act_value_grad<ACT>(__fmul_rn(g[k], gsc), v, dv);
                x[k] = GATED ? d * __fmul_rn(u[k], usc) * dv : d * dv;
                y[k] = d * v;
            }
            dg.w[2 * i] = pack_bf16(x[0], x[1]), dg.w[2 * i + 1] = pack_bf16(x[2], x[3]);
            if (GATED) du.w[2 * i] = pack_bf16(y[0], y[1]), du.w[2 * i + 1] = pack_bf16(y[2], y[3]);
        }
        store_bf16x16(a.dG + wk.row * a.ldg + c, dg, a.v32);
        if (GATED) store_bf16x16(a.dU + wk.row * a.ldu + c, du, a.v32);
    }
}

// RMSNorm backward from the checkpointed input.  With v_k = du_k gain_k,
//   r = (sum x^2 / K + eps)^-1/2,  n_k = x_k r,  m = sum_k v_k n_k / K,
//   dx_k = r (v_k - n_k m) (+ residual gradient),   dgain_k = sum_t du n.
// Neither r^2, r^3 nor x^2 appears on its own: they leave fp32's range long
// before x, r and dx do.  The row's sums are formed from the codes (x = code 2^e)
// next to the largest exponent of the row that has a code other than zero, E:
// sum x^2 = 2^2E s1 and sum v x = 2^E s2 with s1, s2 in range, and what a block
// far below E loses is below the sums' last place.  eps joins them as
// q 2^2Ee, 1/4 <= q < 1, at the larger of E and Ee.
// RT threads share a row, one 16-element chunk each, so both sums are one pass
// over registers and the row is read once; a row longer than
// kNormLongThreads chunks is shared by a cluster of CTAs, which exchange their
// sums.  A CTA takes rows in steps of the grid and keeps its part of dgain in
// registers; the parts meet in shared memory (rows of one CTA, in order) and
// then in norm_dgain_kernel (CTAs, in order), so the result is the same every
// time.
// 16384 x 2048 with the residual gradient: 45 us, 5.2 TB/s: two CTAs an SM (128
// registers a thread) issue 2.6 of 4 instructions a clock while each waits out a
// row's latency and barrier, at 62% of DRAM's rate.  Rows over 8192, with a
// cluster barrier a row: 2.4 TB/s (4096 x 11008).
constexpr int kNormPartials = 640;  // most partial rows of dgain
constexpr int kNormLongThreads = 512;
constexpr int kNormMaxSplit = 8;    // CTAs a row: 8 x 512 chunks of 16 = 65536

struct NormBwdArgs {
    const uint8_t *xc;
    const uint32_t *xs;
    int64_t ldc, rp;
    const uint16_t *gain;  // nullptr: 1
    const uint16_t *dU;
    const uint16_t *dR;    // nullptr: none
    uint16_t *dX;
    float *partial;        // [grid, K]; nullptr: no dgain
    int32_t T, K;
    int32_t v32;           // every bf16 row is 32-byte aligned
    int32_t split;         // CTAs that share a row (a cluster)
    float eps_q;           // eps = eps_q 2^(2 (eps_e - 127))
    int32_t eps_e;
};

// A row's sums so far: sum x^2 = s1 2^(2 (top - 127)), sum v x = s2 2^(top - 127);
// top is a scale byte (0 for nothing but zeros, 255 for a block that is not finite).
struct NormSums {
    float s1, s2;
    int top;
};

// 2^d, 0 below fp32's normal range (d <= 127)
__device__ __forceinline__ float norm_pow2(int d) { return __uint_as_float(static_cast<uint32_t>(max(d + 127, 0)) << 23); }

// `n` (a power of two up to 32) partial sums joined at the largest of their
// exponents: lane l takes part l % n, and a butterfly adds them in one order.
__device__ __forceinline__ NormSums norm_join(const NormSums *p, int n)
{
    NormSums s = p[threadIdx.x & (n - 1)];
    const int top = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(s.top)));
    const float f = norm_pow2(s.top - top);
    s = {s.s1 * f * f, s.s2 * f, top};
#pragma unroll
    for (int off = 1; off < n; off <<= 1) {
        s.s1 += __shfl_xor_sync(0xffffffffu, s.s1, off);
        s.s2 += __shfl_xor_sync(0xffffffffu, s.s2, off);
    }
    return s;
}

template <int TYPE, int RT>
__global__ void __launch_bounds__(RT > 256 ? RT : 256, RT > 256 ? 1 : 2) norm_backward_kernel(NormBwdArgs a)
{
    constexpr int kRows = RT >= 256 ? 1 : 256 / RT;  // rows of one step
    constexpr int W = RT / 32;
    __shared__ NormSums red[2][kRows][W];
    __shared__ NormSums parts[2][kNormMaxSplit];  // a long row: the CTAs' sums
    extern __shared__ float dg_sh[];  // [K]
    grid_wait_and_release();
    // every CTA of a cluster runs before one writes to another's shared memory
    if (RT == kNormLongThreads && a.split > 1) cluster_sync_all();
    const int sub = threadIdx.x / RT, lt = threadIdx.x % RT;
    const int chunks = a.K / 16;
    const int rank = a.split > 1 ? static_cast<int>(blockIdx.x) % a.split : 0;
    const int unit = static_cast<int>(blockIdx.x) / a.split, units = static_cast<int>(gridDim.x) / a.split;
    const int ci = rank * RT + lt;  // this thread's chunk
    const bool mine = ci < chunks;
    const float invk = 1.0f / static_cast<float>(a.K);
    Bf16x16 gain;  // bf16 1.0 where there are none
#pragma unroll
    for (int k = 0; k < 8; ++k) gain.w[k] = 0x3f803f80u;
    if (a.gain && mine) gain = load_bf16x16(a.gain + 16 * ci, false);
    const int blk = ci >> 3;  // scale byte of the chunk's block, without the row's part
    const uint8_t *sbase = reinterpret_cast<const uint8_t *>(a.xs) + 4 * (blk >> 2) * a.rp + (blk & 3);
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.0f;

    // a row as it is read: the next one's loads are in flight while this one
    // is worked on
    uint4 xq;
    Bf16x16 du, dr;
    uint32_t sb;
    auto load = [&](int64_t row) {
        const int64_t r127 = row & 127, rpart = 4 * (row - r127 + 4 * (r127 & 31) + (r127 >> 5));
        xq = make_uint4(0u, 0u, 0u, 0u);
        du = dr = Bf16x16{};
        sb = 127u;
        if (row < a.T && mine) {
            xq = __ldg(reinterpret_cast<const uint4 *>(a.xc + row * a.ldc) + ci);
            du = load_bf16x16(a.dU + row * a.K + 16 * ci, a.v32);
            if (a.dR) dr = load_bf16x16_plain(a.dR + row * a.K + 16 * ci, a.v32);  // dR may be dX
            sb = __ldg(sbase + rpart);
        }
    };
    int parity = 0;
    const int64_t step = static_cast<int64_t>(units) * kRows;
    int64_t base = static_cast<int64_t>(unit) * kRows;
    load(base + sub);
    for (; base < a.T; base += step, parity ^= 1) {
        const int64_t row = base + sub;
        const bool active = row < a.T;
        uint32_t qw[4] = {xq.x, xq.y, xq.z, xq.w};
        // a block of zeros has no exponent (its byte stands for 2^0), one that
        // is not finite the largest
        constexpr uint32_t kMagnitude = TYPE == kB8I8 ? 0xffffffffu : 0x7f7f7f7fu;
        const bool zeros = ((qw[0] | qw[1] | qw[2] | qw[3]) & kMagnitude) == 0u && sb != 255u;
        const int byte = zeros ? 0 : static_cast<int>(sb);
        const Bf16x16 cdu = du, cdr = dr;
        if (base + step < a.T) load(row + step);
        NormSums s = {byte == 255 ? __uint_as_float(0x7fc00000u) : 0.0f, 0.0f, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4];
            b8_decode4<TYPE>(qw[i], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t dw = cdu.w[2 * i + (k >> 1)], gw = gain.w[2 * i + (k >> 1)];
                s.s1 = fmaf(y[k], y[k], s.s1);
                s.s2 = fmaf((k & 1 ? bf16_hi(dw) : bf16_lo(dw)) * (k & 1 ? bf16_hi(gw) : bf16_lo(gw)), y[k], s.s2);
            }
        }
        s.top = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(byte)));
        const float f = norm_pow2(byte - s.top);
        s.s1 *= f * f;
        s.s2 *= f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            s.s1 += __shfl_xor_sync(0xffffffffu, s.s1, off);
            s.s2 += __shfl_xor_sync(0xffffffffu, s.s2, off);
        }
        if constexpr (W > 1) {
            // two buffers in turn: one barrier (of the row's threads) a step
            // suffices
            if ((lt & 31) == 0) red[parity][sub][lt >> 5] = s;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(RT) : "memory");
            s = norm_join(red[parity][sub], W);
        }
        if constexpr (RT == kNormLongThreads) {
            if (a.split > 1) {
                // each CTA's sums to all of the cluster, joined in every CTA
                // alike; again two buffers and one barrier
                if (lt < a.split) {
                    const uint32_t to = map_shared_rank(smem_addr(&parts[parity][rank]), lt);
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "f"(s.s1) : "memory");
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + 4u), "f"(s.s2) : "memory");
                    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + 8u), "r"(s.top) : "memory");
                }
                __syncwarp();
                cluster_sync_all();
                s = norm_join(parts[parity], a.split);
            }
        }
        // mean x^2 + eps = t 2^(2 (e - 127)), at least 2^-252 (r at most 2^126)
        const int e = max(max(s.top, a.eps_e), 1);
        const float g1 = norm_pow2(s.top - e), g2 = norm_pow2(a.eps_e - e);
        float t = fmaf(s.s1 * invk * g1, g1, a.eps_q * g2 * g2);
        if (e == 1) t = fmaxf(t, 1.0f);
        const float rm = rsqrtf(t), r = rm * norm_pow2(127 - e);
        const float m = s.s2 * g1 * rm * invk;
        const float xr = rm * norm_pow2(byte - e);  // n = code xr
        if (!active || !mine) continue;
        Bf16x16 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // decoded again: the values held over the barrier spilled
            asm volatile("" : "+r"(qw[i]));
            float y[4];
            b8_decode4<TYPE>(qw[i], y);
            float out[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t dw = cdu.w[2 * i + (k >> 1)], gw = gain.w[2 * i + (k >> 1)], rw = cdr.w[2 * i + (k >> 1)];
                const float d = k & 1 ? bf16_hi(dw) : bf16_lo(dw), n = y[k] * xr;
                acc[4 * i + k] = fmaf(d, n, acc[4 * i + k]);
                out[k] = fmaf(r, fmaf(-m, n, d * (k & 1 ? bf16_hi(gw) : bf16_lo(gw))), k & 1 ? bf16_hi(rw) : bf16_lo(rw));
            }
            o.w[2 * i] = pack_bf16(out[0], out[1]);
            o.w[2 * i + 1] = pack_bf16(out[2], out[3]);
        }
        store_bf16x16(a.dX + row * a.K + 16 * ci, o, a.v32);
    }
    if (!a.partial) return;
    float *p = kRows > 1 ? dg_sh + 16 * ci : nullptr;
    float4 *o = reinterpret_cast<float4 *>(a.partial + static_cast<int64_t>(unit) * a.K + 16 * ci);
    for (int s = 0; s < kRows; ++s) {
        if (sub == s && mine) {
            if (kRows > 1 && s > 0)
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[k] += p[k];
            if (s == kRows - 1) {
#pragma unroll
                for (int q = 0; q < 4; ++q) o[q] = make_float4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) p[k] = acc[k];
            }
        }
        if (kRows > 1) __syncthreads();
    }
}

// dgain[k] = the sum of n partial rows, in 32 interleaved parts (a warp each)
// joined in order.
__global__ void __launch_bounds__(1024) norm_dgain_kernel(const float *__restrict__ partial, int32_t n, int32_t K,
                                                          float *__restrict__ dgain)
{
    __shared__ float sh[32][33];
    grid_wait_and_release();
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int k = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 4
        for (int i = part; i < n; i += 32) s += partial[static_cast<int64_t>(i) * K + k];
    }
    sh[part][lane] = s;
    __syncthreads();
    if (part == 0 && k < K) {
        s = sh[0][lane];
#pragma unroll
        for (int i = 1; i < 32; ++i) s += sh[i][lane];
        dgain[k] = s;
    }
}

}  // namespace sbl
