// sbl_act_norm.cuh -- RMSNorm fused with the per-token absmax int8 quantiser
// (sbl_act.cuh) on sm_100a, optionally with an 8-bit checkpoint of its input.
#pragma once

#include "sbl_b8_format.cuh"
#include "sbl_b8_device.cuh"

namespace sbl {

constexpr int kActMaxChunks = 8;  // 16-byte chunks (8 bf16) per thread

// Four int8 codes sat8(rint(fl32(x r))) packed LSB first.
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float r)
{
    const uint32_t q0 = rne_byte(__fmul_rn(a, r)), q1 = rne_byte(__fmul_rn(b, r));
    const uint32_t q2 = rne_byte(__fmul_rn(c, r)), q3 = rne_byte(__fmul_rn(d, r));
    uint32_t lo, hi, w;
    asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(lo) : "r"(q0), "r"(q1));
    asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(hi) : "r"(q2), "r"(q3));
    asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(w) : "r"(lo), "r"(hi));
    return w;
}

// u = fl32(fl32(x * r) * g) of one 8-element chunk (g: bf16 gains or none)
__device__ __forceinline__ void norm_chunk(const uint4 &v, const uint16_t *__restrict__ g, int ci, int chunks,
                                           float r, float (&u)[8])
{
    const uint4 gv = (g && ci < chunks) ? __ldg(reinterpret_cast<const uint4 *>(g) + ci) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[2 * i] = __fmul_rn(bf16_lo(w[i]), r);
        u[2 * i + 1] = __fmul_rn(bf16_hi(w[i]), r);
        if (g) {
            u[2 * i] = __fmul_rn(u[2 * i], bf16_lo(gw[i]));
            u[2 * i + 1] = __fmul_rn(u[2 * i + 1], bf16_hi(gw[i]));
        }
    }
}

// RMSNorm fused with the quantiser (the norm before Q_a in forward step 1 of
// the Sparse-BitNet summary): per row, S = sum of x_k^2 in fp64 over the
// pairwise tree of the row in flat order, r = fl32(1 / sqrt(S / K + eps)),
// u_k = fl32(fl32(x_k * r) * g_k) (g: bf16 gains, none = 1), then the
// absmax int8 quantisation of u.
//
// That tree equals the tree of the row padded with +0.0 to 64 RT elements (a
// sum with +0.0 is exact), so it is assembled from aligned subtrees of the
// layout of the plain quantiser: thread lt of a row holds the 8-element
// chunks lt + c RT (slot c < 8; coalesced loads).  Slot c of warp w is the
// aligned 256-element block of chunks c RT + 32 w .. + 31, and slot c of the
// row the aligned block c RT .. (c + 1) RT - 1.  Each chunk is an 8-leaf tree;
// a reduce-scatter over lanes (xor 1, 2, 4: adjacent lanes first, each lane
// keeping half, then a quarter, then one of its slot sums) and two
// butterflies (xor 8, 16) leave in lane L the warp's sum of slot
// 4 (L & 1) + 2 (L >> 1 & 1) + (L >> 2 & 1); the row's first warp then adds
// the warps of each slot pairwise and the slots pairwise.  Every addition
// joins two adjacent aligned subtrees (a + b == b + a exactly).
//
// CK (a b8 type, or kNoCkpt) also writes the b8 checkpoint of X from the held
// chunks: chunks 16 b .. 16 b + 15 are block b and sit in one half warp.  The
// grid then covers the rows padded to 128, whose scales are 127.
constexpr int kNoCkpt = -1;
struct NormCkpt {
    uint8_t *codes;
    uint32_t *scales;
    int64_t rp;
    int32_t words;  // scale words per row
};

//
// NC: 16-byte chunks a thread holds.  With a checkpoint 4 (twice the threads a
// row): the scaled row then fits in registers and is computed once.
template <int RT, int CK = kNoCkpt, int NC = kActMaxChunks>
__global__ void __launch_bounds__(RT > 256 ? RT : 256, RT > 256 ? 1 : 3)
    act_norm_quant_kernel(const uint16_t *__restrict__ X, int32_t T, int32_t K, const uint16_t *__restrict__ g,
                          double eps, int8_t *__restrict__ Xq, float *__restrict__ d, NormCkpt ck)
{
    static_assert(RT >= 32 && (RT & (RT - 1)) == 0, "rows are whole warps, a power of two");
    constexpr int kRowsPerCta = RT >= 256 ? 1 : 256 / RT;
    constexpr int W = RT / 32;                        // warps per row
    constexpr int H = (8 * W + 31) / 32;              // (slot, warp) sums per lane of the combining warp
    __shared__ double wsum[kRowsPerCta][8 * W];       // [slot][warp]
    __shared__ float wmax[kRowsPerCta][W];
    __shared__ float rsh[kRowsPerCta];
    const int sub = threadIdx.x / RT, lt = threadIdx.x % RT;
    const int wr = lt >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerCta + sub;
    if constexpr (CK == kNoCkpt) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
        grid_wait_and_release();
    }
    const bool active = row < T;
    const int chunks = K / 8;

    uint4 v[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ci = lt + c * RT;
        v[c] = make_uint4(0u, 0u, 0u, 0u);
        if (active && ci < chunks) v[c] = __ldg(reinterpret_cast<const uint4 *>(X + row * K) + ci);
    }
    if constexpr (CK != kNoCkpt) {
        uint8_t *sb = reinterpret_cast<uint8_t *>(ck.scales);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int ci = lt + c * RT;
            const uint32_t byte = b8_scale_byte<CK>(half_warp_max(bf16x8_absmax(v[c])) << 16);
            if (active && ci < chunks) {
                *(reinterpret_cast<uint2 *>(ck.codes + row * K) + ci) = b8_encode_bf16x8<CK>(v[c], b8_inv_scale(byte));
                const int blk = ci >> 4;
                if ((ci & 15) == 0) sb[4 * b8_word_index(blk >> 2, ck.rp, row) + (blk & 3)] = static_cast<uint8_t>(byte);
            }
        }
        if (row < ck.rp)  // padding: blocks past the last, or a whole padded row
            for (int b = lt + (active ? (chunks + 15) / 16 : 0); b < 4 * ck.words; b += RT)
                sb[4 * b8_word_index(b >> 2, ck.rp, row) + (b & 3)] = 127;
    }
    double cs[kActMaxChunks];
#pragma unroll
    for (int c = 0; c < kActMaxChunks; ++c) {
        cs[c] = 0.0;  // a slot past the held chunks: +0.0 leaves the tree's sums exact
        if (c >= NC) continue;
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
        double sq[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double lo = static_cast<double>(bf16_lo(w[i])), hi = static_cast<double>(bf16_hi(w[i]));
            sq[2 * i] = lo * lo;  // exact: a bf16 square has at most 16 significant bits
            sq[2 * i + 1] = hi * hi;
        }
        cs[c] = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
    }
    // reduce-scatter over the lanes: keep slots 4 b0 .. 4 b0 + 3, then two of
    // them, then one
    const bool b0 = lane & 1, b1 = (lane >> 1) & 1, b2 = (lane >> 2) & 1;
    double r1[4], r2[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double keep = b0 ? cs[4 + i] : cs[i], give = b0 ? cs[i] : cs[4 + i];
        r1[i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double keep = b1 ? r1[2 + i] : r1[i], give = b1 ? r1[i] : r1[2 + i];
        r2[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
    }
    double r3;
    {
        const double keep = b2 ? r2[1] : r2[0], give = b2 ? r2[0] : r2[1];
        r3 = keep + __shfl_xor_sync(0xffffffffu, give, 4);
    }
    r3 = r3 + __shfl_xor_sync(0xffffffffu, r3, 8);
    r3 = r3 + __shfl_xor_sync(0xffffffffu, r3, 16);
    if (lane < 8) wsum[sub][(4 * b0 + 2 * b1 + b2) * W + wr] = r3;
    __syncthreads();
    if (wr == 0) {
        // value i = h 32 + lane is (slot i / W, warp i % W): warps pairwise
        // within each slot (xor < W), slots pairwise across the lane groups
        // (xor W .. 16; lanes past 8 W hold +0.0), then the H blocks pairwise
        double x[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int i = h * 32 + lane;
            x[h] = i < 8 * W ? wsum[sub][i] : 0.0;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = x[h] + __shfl_xor_sync(0xffffffffu, x[h], off);
#pragma unroll
        for (int step = 1; step < H; step *= 2)
#pragma unroll
            for (int h = 0; h < H; h += 2 * step) x[h] = x[h] + x[h + step];
        if (lane == 0)
            rsh[sub] = __double2float_rn(__ddiv_rn(
                1.0, __dsqrt_rn(__dadd_rn(__ddiv_rn(x[0], static_cast<double>(K)), eps))));
    }
    __syncthreads();
    const float r = rsh[sub];

    // u = fl32(fl32(x * r) * g), computed from the held x in both passes (held
    // itself where a thread has few chunks): max|u| over the row, then the
    // quantised stores
    constexpr bool kKeep = NC <= 4;
    float held[kKeep ? NC : 1][8];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float u[8];
        norm_chunk(v[c], g, lt + c * RT, chunks, r, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            amax = fmaxf(amax, fabsf(u[i]));
            if (kKeep) held[kKeep ? c : 0][i] = u[i];
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (lane == 0) wmax[sub][wr] = amax;
    __syncthreads();
    amax = wmax[sub][0];
#pragma unroll
    for (int w = 1; w < W; ++w) amax = fmaxf(amax, wmax[sub][w]);
    if (!active) return;
    const bool zero = !(amax > 0.0f);
    // with a checkpoint the factor is 127 * (1 / a), two roundings (sbl.h)
    const float rq = zero ? 0.0f : CK == kNoCkpt ? __fdiv_rn(127.0f, amax) : __fmul_rn(127.0f, __frcp_rn(amax));
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int ci = lt + c * RT;
        if (ci >= chunks) continue;
        uint2 out = make_uint2(0u, 0u);
        if (!zero) {
            float u[8];
            if constexpr (kKeep) {
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = held[c][i];
            } else {
                norm_chunk(v[c], g, ci, chunks, r, u);
            }
            out.x = quant4(u[0], u[1], u[2], u[3], rq);
            out.y = quant4(u[4], u[5], u[6], u[7], rq);
        }
        reinterpret_cast<uint2 *>(Xq + row * K)[ci] = out;
    }
    if (lt == 0) d[row] = zero ? 0.0f : __fdiv_rn(amax, 127.0f);
}

}  // namespace sbl
