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
//   r = (sum x^2 / K + eps)^-1/2,  c = r^3 / K sum_k v_k x_k,
//   dx_k = r v_k - c x_k (+ residual gradient),   dgain_k = sum_t du x r.
// RT threads share a row; thread lt holds the 8-element chunks lt + j RT
// (j < NC), so both sums are one pass over registers and the row is read
// once.  A CTA takes rows in steps of the grid and keeps its part of dgain in
// registers; the parts meet in shared memory (rows of one CTA, in order) and
// then in norm_dgain_kernel (CTAs, in order), so the result is the same every
// time.
constexpr int kNormPartials = 640;  // most CTAs that leave a partial dgain

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
    float eps;
};

template <int TYPE, int RT, int NC, bool AHEAD>
__global__ void __launch_bounds__(RT > 256 ? RT : 256, RT > 256 ? 1 : 2) norm_backward_kernel(NormBwdArgs a)
{
    constexpr int kRows = RT >= 256 ? 1 : 256 / RT;  // rows of one step
    constexpr int W = RT / 32;
    __shared__ float2 red[2][kRows][W];
    extern __shared__ float dg_sh[];  // [K]
    grid_wait_and_release();
    const int sub = threadIdx.x / RT, lt = threadIdx.x % RT;
    const int chunks = a.K / 8;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const float invk = 1.0f / static_cast<float>(a.K);
    uint4 gain[NC];  // bf16 1.0 where there are none
    const uint8_t *sbase[NC];  // scale byte of the chunk's block, without the row's part
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int ci = lt + j * RT, blk = ci >> 4;
        gain[j] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        if (a.gain && ci < chunks) gain[j] = __ldg(reinterpret_cast<const uint4 *>(a.gain) + ci);
        sbase[j] = reinterpret_cast<const uint8_t *>(a.xs) + 4 * (blk >> 2) * a.rp + (blk & 3);
    }
    float acc[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[j][k] = 0.0f;

    // a row as it is read; AHEAD: the next one's loads are in flight while this
    // one is worked on (not with 1024 threads, whose 64 registers would spill)
    uint2 xq[NC];
    uint4 du[NC], dr[NC];
    uint32_t sb[NC];
    auto load = [&](int64_t row) {
        const int64_t r127 = row & 127, rpart = 4 * (row - r127 + 4 * (r127 & 31) + (r127 >> 5));
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int ci = lt + j * RT;
            xq[j] = make_uint2(0u, 0u);
            du[j] = dr[j] = z;
            sb[j] = 127u;
            if (row < a.T && ci < chunks) {
                xq[j] = __ldg(reinterpret_cast<const uint2 *>(a.xc + row * a.ldc) + ci);
                du[j] = __ldg(reinterpret_cast<const uint4 *>(a.dU + row * a.K) + ci);
                if (a.dR) dr[j] = *(reinterpret_cast<const uint4 *>(a.dR + row * a.K) + ci);  // dR may be dX
                sb[j] = __ldg(sbase[j] + rpart);
            }
        }
    };
    int parity = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
    if (AHEAD) load(base + sub);
    for (; base < a.T; base += step, parity ^= 1) {
        const int64_t row = base + sub;
        const bool active = row < a.T;
        float x[NC][8];
        uint4 cdu[NC], cdr[NC];
        float s1 = 0.0f, s2 = 0.0f;
        if (!AHEAD) load(row);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            b8_load8<TYPE>(xq[j], b8_scale(sb[j]), x[j]);
            cdu[j] = du[j];
            cdr[j] = dr[j];
        }
        if (AHEAD && base + step < a.T) load(row + step);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float d[8], g[8];
            unpack_bf16x8(cdu[j], d);
            unpack_bf16x8(gain[j], g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s1 = fmaf(x[j][k], x[j][k], s1);
                s2 = fmaf(d[k] * x[j][k], g[k], s2);
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            s1 += __shfl_xor_sync(0xffffffffu, s1, off);
            s2 += __shfl_xor_sync(0xffffffffu, s2, off);
        }
        if constexpr (W > 1) {
            // two buffers in turn: one barrier (of the row's threads) a step
            // suffices
            if ((lt & 31) == 0) red[parity][sub][lt >> 5] = make_float2(s1, s2);
            asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "n"(RT) : "memory");
            s1 = s2 = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 p = red[parity][sub][w];
                s1 += p.x;
                s2 += p.y;
            }
        }
        const float r = rsqrtf(s1 * invk + a.eps);
        const float c = r * r * r * (s2 * invk);
        if (!active) continue;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int ci = lt + j * RT;
            if (ci >= chunks) continue;
            float d[8], g[8], e[8], o[8];
            unpack_bf16x8(cdu[j], d);
            unpack_bf16x8(gain[j], g);
            unpack_bf16x8(cdr[j], e);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                acc[j][k] = fmaf(d[k] * x[j][k], r, acc[j][k]);
                o[k] = fmaf(d[k], r * g[k], fmaf(-c, x[j][k], e[k]));
            }
            *(reinterpret_cast<uint4 *>(a.dX + row * a.K) + ci) = pack_bf16x8(o);
        }
    }
    if (!a.partial) return;
    for (int s = 0; s < kRows; ++s) {
        if (sub == s) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int ci = lt + j * RT;
                if (ci >= chunks) continue;
                float *p = kRows > 1 ? dg_sh + 8 * ci : nullptr;
                float *o = a.partial + static_cast<int64_t>(blockIdx.x) * a.K + 8 * ci;
                if (kRows > 1 && s > 0)
#pragma unroll
                    for (int k = 0; k < 8; ++k) acc[j][k] += p[k];
                if (s == kRows - 1) {
                    reinterpret_cast<float4 *>(o)[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
                    reinterpret_cast<float4 *>(o)[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) p[k] = acc[j][k];
                }
            }
        }
        __syncthreads();
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
