// sbl_b8_format.cuh -- the 8-bit block format ("b8"): scales, codes and layout.
//
// A b8 matrix [R, C] stores 8-bit codes (e4m3, e5m2 or int8) and one power of
// two 2^e per block of 128 codes along a row (or one for a 128 x 128 tile).
//   a = max |x| over the block,  e = the smallest integer >= -126 with
//   a <= MAX 2^e (MAX = 448, 57344, 127; e = 0 when a == 0),
//   code = round_half_even_to_type(x 2^-e).
// The scaling by 2^-e is exact, so a code is ONE rounding of x and every
// result is defined bit for bit, whatever computes it.  e is stored as the
// byte e + 127, the type the block-scaled tensor-core MMA reads; 255 marks a
// block that held an Inf or a NaN and decodes to NaN.
//
// Scale bytes: four consecutive blocks of a row make a 32-bit word (block
// 4w + i in byte i); the words of word column w are contiguous over rows,
// 128 rows at a time in the order row -> 4 (row % 32) + (row % 128) / 32, which
// is the order in which tcgen05.cp (32x128b) spreads 128 rows over tensor
// memory lanes and columns.  Rows are padded to 128 and blocks to 4 with 127.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace sbl {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Round-half-even of |v| < 2^22 by the fp32 adder: fl(v + 1.5 2^23) has ulp 1
// and lies in [2^23, 2^24), so its bits are 0x4B400000 + rint(v), and the low
// byte is rint(v) as an int8 bit pattern when rint(v) is in [-128, 127].  The
// quantisers' products are at most 127 but for their roundings, for |x| <= a:
// |fl32(x fl32(127 / a))| <= 127 (1 + 2^-24)^2, with the checkpointed norm's
// factor |fl32(x fl32(127 fl32(1 / a)))| <= 127 (1 + 2^-24)^3, and a b8 int8 code's
// x 2^-e is exact.  So rint lies in [-127, 127] and the clamp to [-128, 127] never
// binds; one FADD replaces the float-to-int conversion.
__device__ __forceinline__ uint32_t rne_byte(float v)
{
    return __float_as_uint(__fadd_rn(v, 12582912.0f));
}

enum B8Type : int { kB8E4M3 = 0, kB8E5M2 = 1, kB8I8 = 2 };
enum B8Source : int { kSrcBf16 = 0, kSrcF32 = 1, kSrcB8 = 2 };

constexpr uint32_t kB8PadWord = 0x7f7f7f7fu;  // four scales of 2^0
constexpr uint32_t kF32Inf = 0x7f800000u;

// Index of a row's scale word inside word column w of a matrix whose rows are
// padded to rp (a multiple of 128).
__host__ __device__ __forceinline__ int64_t b8_word_index(int64_t w, int64_t rp, int64_t row)
{
    const int64_t r = row & 127;
    return w * rp + (row - r) + 4 * (r & 31) + (r >> 5);
}

// The scale byte for a block whose largest magnitude has the fp32 bits `a`.
// With MAX = (1 + top / 2^23) 2^shift the exponent is a's own less shift, and one
// more when a's fraction exceeds top: adding 2^23 - 1 - top carries exactly then.
template <int TYPE>
__device__ __forceinline__ uint32_t b8_scale_byte(uint32_t a)
{
    constexpr int shift = TYPE == kB8E4M3 ? 8 : TYPE == kB8E5M2 ? 15 : 6;
    constexpr int top = TYPE == kB8I8 ? 0x7e0000 : 0x600000;
    constexpr int add = 0x7fffff - top - (shift << 23);
    const int e = max(static_cast<int>(a) + add, 1 << 23) >> 23;
    return a >= kF32Inf ? 255u : a == 0u ? 127u : static_cast<uint32_t>(e);
}

// 2^-(byte - 127), exact; 0 for a block that is not finite (its codes are 0)
__device__ __forceinline__ float b8_inv_scale(uint32_t byte)
{
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127): NaN for 255, 2^-127 (subnormal) for 0
__device__ __forceinline__ float b8_scale(uint32_t byte)
{
    const uint32_t bits = byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23;
    return __uint_as_float(bits);
}

// Four codes of already scaled values, lowest address first.
template <int TYPE>
__device__ __forceinline__ uint32_t b8_encode4(float a, float b, float c, float d)
{
    if constexpr (TYPE == kB8I8) {
        const uint32_t q0 = rne_byte(a), q1 = rne_byte(b), q2 = rne_byte(c), q3 = rne_byte(d);
        return __byte_perm(__byte_perm(q0, q1, 0x0040), __byte_perm(q2, q3, 0x0040), 0x5410);
    } else {
        constexpr __nv_fp8_interpretation_t f = TYPE == kB8E4M3 ? __NV_E4M3 : __NV_E5M2;
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, f);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, f);
        return lo | (hi << 16);
    }
}

// Four codes of values still to be scaled by inv = 2^-e.  int8: the product
// is exact, so it may be fused with the rounding addition.
template <int TYPE>
__device__ __forceinline__ uint32_t b8_scale_encode4(float a, float b, float c, float d, float inv)
{
    if constexpr (TYPE == kB8I8) {
        const float m = 12582912.0f;  // see rne_byte
        const uint32_t q0 = __float_as_uint(__fmaf_rn(a, inv, m)), q1 = __float_as_uint(__fmaf_rn(b, inv, m));
        const uint32_t q2 = __float_as_uint(__fmaf_rn(c, inv, m)), q3 = __float_as_uint(__fmaf_rn(d, inv, m));
        return __byte_perm(__byte_perm(q0, q1, 0x0040), __byte_perm(q2, q3, 0x0040), 0x5410);
    } else {
        return b8_encode4<TYPE>(__fmul_rn(a, inv), __fmul_rn(b, inv), __fmul_rn(c, inv), __fmul_rn(d, inv));
    }
}

// The values (unscaled) of the four codes of a word.
template <int TYPE>
__device__ __forceinline__ void b8_decode4(uint32_t w, float (&v)[4])
{
    if constexpr (TYPE == kB8I8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(static_cast<int8_t>((w >> (8 * i)) & 0xffu));
    } else {
        constexpr __nv_fp8_interpretation_t f = TYPE == kB8E4M3 ? __NV_E4M3 : __NV_E5M2;
        const __half2 lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), f);
        const __half2 hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), f);
        const float2 a = __half22float2(lo), b = __half22float2(hi);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
}

// Largest |x| of eight bf16 values as bf16 bits (magnitudes of bf16 order
// like their bits; a NaN orders above Inf).
__device__ __forceinline__ uint32_t bf16x8_absmax(const uint4 &v)
{
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffffu, m >> 16);
}

// Eight bf16 values quantised with the factor inv (0: a block that is not
// finite, codes 0).
template <int TYPE>
__device__ __forceinline__ uint2 b8_encode_bf16x8(const uint4 &v, float inv)
{
    const uint2 w = make_uint2(b8_scale_encode4<TYPE>(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), inv),
                               b8_scale_encode4<TYPE>(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), inv));
    return inv == 0.0f ? make_uint2(0u, 0u) : w;
}

// How the element-wise kernels walk a matrix (no division: a 64-bit one costs
// as much as the work on six elements).  per_warp > 0: warp v of a CTA takes row
// 8 blockIdx.x + v and the scale words [w0, w1) of it (512 columns each).
// per_warp == 0, for rows of many words: the CTA takes row blockIdx.x, its warps
// the words v, v + 8, ..., so that it streams through one stretch of memory.
struct B8Walk {
    int64_t row;
    int w0, w1, step;
};

__device__ __forceinline__ B8Walk b8_walk(int words, int per_warp)
{
    const int v = threadIdx.x >> 5;
    if (per_warp == 0) return {static_cast<int64_t>(blockIdx.x), v, words, 8};
    const int w0 = static_cast<int>(blockIdx.y) * per_warp;
    return {static_cast<int64_t>(blockIdx.x) * 8 + v, w0, min(w0 + per_warp, words), 1};
}

// Sixteen bf16 of a row, one lane's share in the element-wise kernels: 32-byte
// accesses where every row is 32-byte aligned (v32), pairs of 16-byte ones
// otherwise.
struct Bf16x16 {
    uint32_t w[8];
};

__device__ __forceinline__ Bf16x16 load_bf16x16(const uint16_t *p, bool v32)
{
    Bf16x16 r;
    if (v32) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    }
    return r;
}

// The same from memory that this kernel may also write.
__device__ __forceinline__ Bf16x16 load_bf16x16_plain(const uint16_t *p, bool v32)
{
    Bf16x16 r;
    if (v32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    }
    return r;
}

__device__ __forceinline__ void store_bf16x16(uint16_t *p, const Bf16x16 &r, bool v32)
{
    if (v32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
                     "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    }
}

// Largest |x| as bf16 bits, as bf16x8_absmax.
__device__ __forceinline__ uint32_t bf16x16_absmax(const Bf16x16 &v)
{
    uint32_t m = v.w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, v.w[i] & 0x7fff7fffu);
    return max(m & 0xffffu, m >> 16);
}

// Sixteen codes with the factor inv (0: a block that is not finite, codes 0).
template <int TYPE>
__device__ __forceinline__ uint4 b8_encode_bf16x16(const Bf16x16 &v, float inv)
{
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        q[i] = b8_scale_encode4<TYPE>(bf16_lo(v.w[2 * i]), bf16_hi(v.w[2 * i]), bf16_lo(v.w[2 * i + 1]), bf16_hi(v.w[2 * i + 1]), inv);
    return inv == 0.0f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(q[0], q[1], q[2], q[3]);
}

// max over the 8 lanes that hold a block (sixteen values each)
__device__ __forceinline__ uint32_t eighth_max(uint32_t v)
{
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// The same for two 16-bit magnitudes at once.
__device__ __forceinline__ uint32_t eighth_max2(uint32_t v)
{
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) v = __vmaxu2(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// The warp's scale word from its four blocks' bytes (lanes 8 b .. hold block b's).
__device__ __forceinline__ uint32_t scale_word(uint32_t byte, int lane)
{
    uint32_t w = byte << (8 * (lane >> 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    return w | __shfl_xor_sync(0xffffffffu, w, 16);
}

// max over the 16 lanes of a half warp
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v)
{
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Eight codes of one block decoded with its scale s = 2^e.
template <int TYPE>
__device__ __forceinline__ void b8_load8(const uint2 &q, float s, float (&v)[8])
{
    float lo[4], hi[4];
    b8_decode4<TYPE>(q.x, lo);
    b8_decode4<TYPE>(q.y, hi);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul_rn(lo[k], s), v[4 + k] = __fmul_rn(hi[k], s);
}

}  // namespace sbl
