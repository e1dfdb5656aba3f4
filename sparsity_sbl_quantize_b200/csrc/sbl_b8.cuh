// sbl_b8.cuh -- quantiser, transposer and reader of b8 matrices (the format:
// sbl_b8_format.cuh) on sm_100a.
#pragma once

#include "sbl_b8_format.cuh"
#include "sbl_b8_device.cuh"

namespace sbl {

// ------------------------------------------------------------ row blocks --
// One warp per (row, 512 columns): lane l holds the sixteen values at columns
// 16 l .., eight lanes a block, and the warp writes one scale word.  What is done
// once per block is thus shared by sixteen values a lane (with eight, the
// int8 gated activation below spent a quarter of its instructions on it).
// Memory bound: 16384 x 11008 at the copy rate.
struct B8RowArgs {
    const void *X;
    int64_t ldx;        // elements
    int32_t rows, cols;
    uint8_t *codes;
    int64_t ldc;        // bytes, >= cols
    uint32_t *scales;
    int64_t rp;         // rows padded to 128
    int32_t words;      // scale words per row
    int32_t per_warp;   // of which a warp takes so many
    int32_t v32;        // bf16 rows are 32-byte aligned
};

template <int TYPE, int SRC>
__global__ void __launch_bounds__(256) b8_quantize_rows_kernel(B8RowArgs a)
{
    grid_wait_and_release();
    const int lane = threadIdx.x & 31;
    const B8Walk u = b8_walk(a.words, a.per_warp);
    if (u.row >= a.rp) return;
    uint32_t *scales = a.scales + b8_word_index(0, a.rp, u.row);
    if (u.row >= a.rows) {
        if (lane == 0)
            for (int w = u.w0; w < u.w1; w += u.step) scales[w * a.rp] = kB8PadWord;
        return;
    }
    uint8_t *codes = a.codes + u.row * a.ldc;
    for (int w = u.w0; w < u.w1; w += u.step) {
        const int c = 512 * w + 16 * lane;
        const bool ok = c < a.cols;
        uint32_t byte;
        uint4 q;
        if constexpr (SRC == kSrcBf16) {
            Bf16x16 v = {};
            if (ok) v = load_bf16x16(static_cast<const uint16_t *>(a.X) + u.row * a.ldx + c, a.v32);
            byte = b8_scale_byte<TYPE>(eighth_max(bf16x16_absmax(v)) << 16);
            q = b8_encode_bf16x16<TYPE>(v, b8_inv_scale(byte));
        } else {
            float4 v[4];
            const float4 *x = reinterpret_cast<const float4 *>(static_cast<const float *>(a.X) + u.row * a.ldx + c);
            uint32_t m = 0;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v[h] = ok ? __ldg(x + h) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                m = max(m, max(max(__float_as_uint(v[h].x) & 0x7fffffffu, __float_as_uint(v[h].y) & 0x7fffffffu),
                               max(__float_as_uint(v[h].z) & 0x7fffffffu, __float_as_uint(v[h].w) & 0x7fffffffu)));
            }
            byte = b8_scale_byte<TYPE>(eighth_max(m));
            const float inv = b8_inv_scale(byte);
            uint32_t p[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) p[h] = b8_scale_encode4<TYPE>(v[h].x, v[h].y, v[h].z, v[h].w, inv);
            q = inv == 0.0f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(p[0], p[1], p[2], p[3]);
        }
        if (ok) *reinterpret_cast<uint4 *>(codes + c) = q;
        const uint32_t word = scale_word(byte, lane);
        if (lane == 0) scales[w * a.rp] = word;
    }
}

// Codes and scales back to bf16 (one rounding of code 2^e, exact unless the
// value lies below bf16's normal range).  The layout of the quantiser.
struct B8ReadArgs {
    const uint8_t *codes;
    int64_t ldc;
    const uint32_t *scales;
    int64_t rp;
    int32_t rows, cols, words, per_warp, v32;
    uint16_t *X;
    int64_t ldx;
};

template <int TYPE>
__global__ void __launch_bounds__(256) b8_dequantize_kernel(B8ReadArgs a)
{
    grid_wait_and_release();
    const int lane = threadIdx.x & 31;
    const B8Walk u = b8_walk(a.words, a.per_warp);
    if (u.row >= a.rows) return;
    const uint32_t *scales = a.scales + b8_word_index(0, a.rp, u.row);
    for (int w = u.w0; w < u.w1; w += u.step) {
        const int c = 512 * w + 16 * lane;
        if (c >= a.cols) continue;
        const float s = b8_scale((__ldg(scales + w * a.rp) >> (8 * (lane >> 3))) & 0xffu);
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a.codes + u.row * a.ldc + c));
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
        Bf16x16 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
            b8_decode4<TYPE>(qw[i], v);
            r.w[2 * i] = pack_bf16(__fmul_rn(v[0], s), __fmul_rn(v[1], s));
            r.w[2 * i + 1] = pack_bf16(__fmul_rn(v[2], s), __fmul_rn(v[3], s));
        }
        store_bf16x16(a.X + u.row * a.ldx + c, r, a.v32);
    }
}

// ------------------------------------------------------ tiles, transposed --
// One CTA per 128 x 128 tile; thread (rg, cg) holds the 8 x 8 values at rows
// 8 rg .., columns 8 cg .. as they were read (decoded anew where needed: the
// registers that this frees hold more loads in flight), so a row block is the 16
// lanes of a half warp, a column block is 16 threads of one cg, and a
// thread's column of eight is eight consecutive bytes of the transposed row.
// Both orders come from one read of X; the transposed bytes pass through a
// 16 KiB swizzled tile so that both outputs are written 128 bytes at a time.
//
// out   the row blocks (codes nullptr: not written)
// out_t the same matrix transposed, [cols, rows] (codes nullptr: not written)
// TILES: one scale per 128 x 128 tile for both.  The transpose is then exact;
// otherwise its blocks run along the rows of X and have scales of their own.
struct B8TileArgs {
    const void *X;      // bf16, fp32 or b8 codes
    int64_t ldx;        // elements (bytes of a b8 row)
    const uint32_t *xs; // b8 source: its scales
    int64_t xrp;
    int32_t rows, cols;
    uint8_t *codes;
    int64_t ldc;
    uint32_t *scales;
    int64_t rp;
    uint8_t *codes_t;
    int64_t ldt;        // round_up(rows, 16)
    uint32_t *scales_t;
    int64_t rpt;        // cols padded to 128
    int32_t tiles_c;    // column tiles; the grid runs over tiles, columns fastest
    int32_t late;       // nothing here depends on the kernel before (sbl_b8_device.cuh)
};

template <int TYPE, int SRC, int SRC_TYPE, bool TILES>
__global__ void __launch_bounds__(256, SRC == kSrcF32 ? 2 : 4) b8_tile_kernel(B8TileArgs a)
{
    __shared__ __align__(16) uint8_t tile[128 * 128];
    // a thread row's column maxima: two bf16 magnitudes a word, or fp32 bits
    constexpr int kMaxWords = SRC == kSrcBf16 ? 64 : 128;
    __shared__ __align__(16) uint32_t colmax[16][kMaxWords];
    __shared__ uint32_t wmax[8];
    __shared__ __align__(16) uint8_t rbyte[128], cbyte[128];
    if (!a.late) grid_wait_and_release();
    const int tid = threadIdx.x, lane = tid & 31;
    const int rg = tid >> 4, cg = tid & 15;
    const int tr = static_cast<int>(blockIdx.x) / a.tiles_c;
    const int r0 = tr * 128, c0 = (static_cast<int>(blockIdx.x) - tr * a.tiles_c) * 128;
    const int col = c0 + 8 * cg;
    const bool col_ok = col < a.cols;
    const int row = r0 + 8 * rg;  // the thread's first row

    // the thread's values as they were read; past L1, which a kernel that has
    // not waited must not trust (and which has nothing to offer here)
    uint4 q[SRC == kSrcBf16 ? 8 : 1];
    float4 f[SRC == kSrcF32 ? 8 : 1][2];
    uint2 b[SRC == kSrcB8 ? 8 : 1];
    __shared__ __align__(16) float rscale[SRC == kSrcB8 ? 128 : 4];  // 2^e of the source's rows
    __shared__ uint32_t rlimits[8];                                  // largest, smallest scale byte of each 32 rows
    if constexpr (SRC == kSrcB8) {
        const int blk = c0 >> 7;
        if (tid < 128) {
            const bool in = r0 + tid < a.rows;
            const uint32_t byte =
                in ? __ldcg(reinterpret_cast<const uint8_t *>(a.xs + b8_word_index(blk >> 2, a.xrp, r0 + tid)) + (blk & 3)) : 0u;
            rscale[tid] = in ? b8_scale(byte) : 1.0f;
            const uint32_t top = __reduce_max_sync(0xffffffffu, byte), low = __reduce_min_sync(0xffffffffu, in ? byte : 255u);
            if (lane == 0) rlimits[tid >> 5] = top, rlimits[4 + (tid >> 5)] = low;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool ok = col_ok && row + i < a.rows;
        const int64_t at = static_cast<int64_t>(row + i) * a.ldx + col;
        if constexpr (SRC == kSrcBf16) {
            q[i] = ok ? __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.X) + at)) : make_uint4(0u, 0u, 0u, 0u);
        } else if constexpr (SRC == kSrcF32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.X) + at);
            const float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            f[i][0] = ok ? __ldcg(p) : z;
            f[i][1] = ok ? __ldcg(p + 1) : z;
        } else {
            b[i] = ok ? __ldcg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.X) + at)) : make_uint2(0u, 0u);
        }
    }
    if constexpr (SRC == kSrcB8) __syncthreads();
    // element j of row i, the eight of row i
    auto row_values = [&](int i, float(&v)[8]) {
        if constexpr (SRC == kSrcBf16) {
            const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(w[j]), v[2 * j + 1] = bf16_hi(w[j]);
        } else if constexpr (SRC == kSrcF32) {
            v[0] = f[i][0].x, v[1] = f[i][0].y, v[2] = f[i][0].z, v[3] = f[i][0].w;
            v[4] = f[i][1].x, v[5] = f[i][1].y, v[6] = f[i][1].z, v[7] = f[i][1].w;
        } else {
            b8_load8<SRC_TYPE>(b[i], rscale[8 * rg + i], v);
        }
    };
    // the staged tile and the column scales to out_t
    auto store_transposed = [&]() {
        __syncthreads();
        // rows past the last are zero codes, so whole 16-byte chunks are
        // written up to the padded row length
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int k = p * 256 + tid;
            const int tc = k >> 3, ch = k & 7;
            const int64_t trow = c0 + tc;
            if (trow < a.cols && r0 + 16 * ch < a.ldt)
                *reinterpret_cast<uint4 *>(a.codes_t + trow * a.ldt + r0 + 16 * ch) =
                    *reinterpret_cast<const uint4 *>(tile + tc * 128 + ((ch ^ ((tc >> 3) & 7)) << 4));
        }
        if (tid < 128) {
            const int64_t trow = c0 + tid;
            const int blk = r0 >> 7, nblk = (a.rows + 127) >> 7;
            uint8_t *p = reinterpret_cast<uint8_t *>(a.scales_t + b8_word_index(blk >> 2, a.rpt, trow));
            p[blk & 3] = trow < a.cols ? cbyte[tid] : 127;
            if (blk == nblk - 1)
                for (int k = (blk & 3) + 1; k < 4; ++k) p[k] = 127;
        }
    };
    // e4m3 to e4m3, the transposed copy alone: in half precision and two columns
    // at a time (below) when the rows' scales lie within 2^5 of one another, as
    // a checkpoint's do.  A code is at most 4 bits wide and at least 2^-9, so
    // code 2^(e - top) is a normal half and exact, and so is its multiple
    // 2^(top - e_column) up to 2^15 (16384 x 11008: 88 us against 99).
    constexpr bool kHalfPath = SRC == kSrcB8 && SRC_TYPE == kB8E4M3 && TYPE == kB8E4M3 && !TILES;
    if constexpr (kHalfPath) {
        const uint32_t top = max(max(rlimits[0], rlimits[1]), max(rlimits[2], rlimits[3]));
        const uint32_t low = min(min(rlimits[4], rlimits[5]), min(rlimits[6], rlimits[7]));
        if (top < 255u && top - low <= 5u) {
            __half2 hs[8][4];
            uint4 m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // 2^(e - top) from the row's 2^e: the difference of the biased exponents
                const uint32_t byte = row + i < a.rows ? __float_as_uint(rscale[8 * rg + i]) >> 23 : top;
                const uint32_t f = (15u + byte - top) << 10;
                const __half2 f2 = __half2_raw{static_cast<unsigned short>(f), static_cast<unsigned short>(f)};
                const uint32_t w[4] = {b[i].x & 0xffffu, b[i].x >> 16, b[i].y & 0xffffu, b[i].y >> 16};
                uint32_t q2[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    hs[i][p] = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[p]), __NV_E4M3)), f2);
                    q2[p] = *reinterpret_cast<const uint32_t *>(&hs[i][p]) & 0x7fff7fffu;
                }
                m.x = __vmaxu2(m.x, q2[0]), m.y = __vmaxu2(m.y, q2[1]), m.z = __vmaxu2(m.z, q2[2]), m.w = __vmaxu2(m.w, q2[3]);
            }
            *reinterpret_cast<uint4 *>(&colmax[rg][4 * cg]) = m;
            __syncthreads();
            bool wide = false;  // a column too far below the tile's top
            if (tid < 64) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) w = __vmaxu2(w, colmax[i][tid]);
                const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                const float st = b8_scale(top);
                const uint32_t b0 = b8_scale_byte<TYPE>(__float_as_uint(__fmul_rn(v.x, st)));
                const uint32_t b1 = b8_scale_byte<TYPE>(__float_as_uint(__fmul_rn(v.y, st)));
                cbyte[2 * tid] = static_cast<uint8_t>(b0);
                cbyte[2 * tid + 1] = static_cast<uint8_t>(b1);
                wide = (v.x != 0.0f && top - b0 > 15u) || (v.y != 0.0f && top - b1 > 15u);
            }
            if (!__syncthreads_or(wide)) {
                const uint2 cb = *reinterpret_cast<const uint2 *>(cbyte + 8 * cg);
                __half2 cf[4];  // 2^(top - e_column); an empty column (codes 0) may take any factor
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const uint32_t pair = (p < 2 ? cb.x : cb.y) >> (16 * (p & 1));
                    const uint32_t d0 = top - (pair & 0xffu), d1 = top - ((pair >> 8) & 0xffu);
                    cf[p] = __half2_raw{static_cast<unsigned short>((15u + (d0 > 15u ? 0u : d0)) << 10),
                                        static_cast<unsigned short>((15u + (d1 > 15u ? 0u : d1)) << 10)};
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        uint32_t r[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            r[i] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hmul2(hs[4 * h + i][p], cf[p])), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t t01 = r[0] | (r[1] << 16), t23 = r[2] | (r[3] << 16);
                        uint8_t *at = tile + (8 * cg + 2 * p) * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + 8 * (rg & 1) + 4 * h;
                        *reinterpret_cast<uint32_t *>(at) = __byte_perm(t01, t23, 0x6420);
                        *reinterpret_cast<uint32_t *>(at + 128) = __byte_perm(t01, t23, 0x7531);
                    }
                store_transposed();
                if (a.late) grid_wait_and_release();
                return;
            }
        }
    }
    auto mag = [](float x) { return __float_as_uint(x) & 0x7fffffffu; };
    auto row_max = [&](int i) {
        if constexpr (SRC == kSrcBf16) {
            return bf16x8_absmax(q[i]) << 16;
        } else {
            float v[8];
            row_values(i, v);
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, mag(v[j]));
            return m;
        }
    };

    // ------------------------------------------------------- block scales
    if constexpr (TILES) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, row_max(i));
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) wmax[tid >> 5] = m;
        __syncthreads();
        m = wmax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, wmax[i]);
        const uint32_t byte = b8_scale_byte<TYPE>(m);
        if (tid < 128) rbyte[tid] = cbyte[tid] = static_cast<uint8_t>(byte);
    } else {
        if (a.codes) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t byte = b8_scale_byte<TYPE>(half_warp_max(row_max(i)));
                if (cg == 0) rbyte[8 * rg + i] = static_cast<uint8_t>(byte);
            }
        }
        if (a.codes_t) {
            if constexpr (SRC == kSrcBf16) {
                uint4 m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m.x = __vmaxu2(m.x, q[i].x & 0x7fff7fffu);
                    m.y = __vmaxu2(m.y, q[i].y & 0x7fff7fffu);
                    m.z = __vmaxu2(m.z, q[i].z & 0x7fff7fffu);
                    m.w = __vmaxu2(m.w, q[i].w & 0x7fff7fffu);
                }
                *reinterpret_cast<uint4 *>(&colmax[rg][4 * cg]) = m;
                __syncthreads();
                if (tid < 64) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) w = __vmaxu2(w, colmax[i][tid]);
                    cbyte[2 * tid] = static_cast<uint8_t>(b8_scale_byte<TYPE>(w << 16));
                    cbyte[2 * tid + 1] = static_cast<uint8_t>(b8_scale_byte<TYPE>(w & 0xffff0000u));
                }
            } else {
                uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v[8];
                    row_values(i, v);
#pragma unroll
                    for (int j = 0; j < 8; ++j) m[j] = max(m[j], mag(v[j]));
                }
                // the two halves apart, so that a quarter warp's 16-byte stores
                // fall on different banks
                *reinterpret_cast<uint4 *>(&colmax[rg][4 * cg]) = make_uint4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<uint4 *>(&colmax[rg][(kMaxWords / 2 + 4 * cg) % kMaxWords]) = make_uint4(m[4], m[5], m[6], m[7]);
                __syncthreads();
                if (tid < 128) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) w = max(w, colmax[i][tid % kMaxWords]);
                    cbyte[8 * ((tid & 63) >> 2) + 4 * (tid >> 6) + (tid & 3)] = static_cast<uint8_t>(b8_scale_byte<TYPE>(w));
                }
            }
        }
    }
    __syncthreads();

    // ----------------------------------------------------------- row codes
    if (a.codes) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!col_ok || row + i >= a.rows) continue;
            const float inv = b8_inv_scale(rbyte[8 * rg + i]);
            float v[8];
            row_values(i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], inv);
            uint2 w = make_uint2(b8_encode4<TYPE>(v[0], v[1], v[2], v[3]), b8_encode4<TYPE>(v[4], v[5], v[6], v[7]));
            if (inv == 0.0f) w = make_uint2(0u, 0u);  // the block is not finite
            *reinterpret_cast<uint2 *>(a.codes + static_cast<int64_t>(row + i) * a.ldc + col) = w;
        }
        // the tile's column of scale bytes (padded rows: 127; a word's blocks
        // past the last column are filled by the last block's tile)
        if (tid < 128) {
            const int64_t srow = r0 + tid;
            const int blk = c0 >> 7, nblk = (a.cols + 127) >> 7;
            uint8_t *p = reinterpret_cast<uint8_t *>(a.scales + b8_word_index(blk >> 2, a.rp, srow));
            p[blk & 3] = srow < a.rows ? rbyte[tid] : 127;
            if (blk == nblk - 1)
                for (int k = (blk & 3) + 1; k < 4; ++k) p[k] = 127;
        }
    }
    // ---------------------------------------------------- transposed codes
    if (a.codes_t) {
        // eight bytes (rows 8 rg ..) of transposed row 8 cg + j, the 16-byte
        // chunk rg / 2 at position (rg / 2) ^ (cg % 8): scaled and encoded
        // four rows at a time, a column's four codes in one word
        const uint2 cb = *reinterpret_cast<const uint2 *>(cbyte + 8 * cg);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) row_values(4 * h + i, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float inv = b8_inv_scale(((j < 4 ? cb.x : cb.y) >> (8 * (j & 3))) & 0xffu);
                uint32_t w = b8_encode4<TYPE>(__fmul_rn(v[0][j], inv), __fmul_rn(v[1][j], inv), __fmul_rn(v[2][j], inv),
                                              __fmul_rn(v[3][j], inv));
                if (inv == 0.0f) w = 0u;
                *reinterpret_cast<uint32_t *>(tile + (8 * cg + j) * 128 + (((rg >> 1) ^ (cg & 7)) << 4) + 8 * (rg & 1) + 4 * h) = w;
            }
        }
        store_transposed();
    }
    if (a.late) grid_wait_and_release();
}

}  // namespace sbl
