// sbl_b8_gemm.cuh -- matrix product of two b8 matrices on the block-scaled
// tensor cores of sm_100a.
//
//   D[m, n] (+)= sum_k 2^(ea[m, k / 128] + eb[n, k / 128]) a[m, k] b[n, k]
//
// a, b: e4m3 or e5m2 codes, K-major; ea, eb: the blocks' exponents.  The MMA
// (tcgen05.mma kind::mxf8f6f4) takes one power-of-two scale per 32 codes from
// tensor memory and applies it before the fp32 accumulation, so a scale per
// 128 costs nothing: the four MMAs of a 128-wide stage name the same scale
// byte (the scale-factor id of the instruction descriptor = block % 4), and
// one 512-byte copy of scale words (tcgen05.cp 32x128b.warpx4, 128 rows x 4
// blocks) serves four stages.  Had the scales been arbitrary fp32 numbers,
// every stage's partial sum would have to leave tensor memory to be scaled in
// registers: 64 FMAs and TMEM reads per SM and clock beside the MMAs.
//
// Tiles are 128 x BN (256, or 128 where that spreads a small product over more
// SMs); roles as in the other tcgen05 products: warp 0 TMA loads, warp 1 MMAs,
// warps 2-9 the epilogue.  CTA pairs with 256 x 256 tiles were built first and
// gave way to this (m x n x k, here and below: 16384 x 11008 x 2048: 309 us against
// 299, 16384 x 2048 x 11008: 296 against 269).  That was no comparison on equal terms: the pair kernel issued
// from a lane-0 branch and copied scales one word at a time, which cost the
// single-CTA kernel 5% and more (below).  Pairs with an elected lane and two-word
// copies have not been measured.
//
// 16384 x 2048 x 11008 takes 269 us in short runs, 2.7 PFLOP/s (84% of twice the
// measured burst bf16 rate, cuBLAS's); the same MMAs without loads or scales take
// 232: the rest is the tensor core waiting between stages and tiles (active 67% of
// the cycles at 8192 x 11008 x 2048).  In a loop of seconds the power limit takes
// another 12%, as it takes 14% of cuBLAS's bf16 product.
#pragma once

#include <cuda_bf16.h>

#include "sbl_b8_format.cuh"
#include "sbl_b8_device.cuh"
#include "sbl_gemm.cuh"  // tile raster, role sizes

namespace sbl {

struct B8GemmArgs {
    int32_t M, N;
    int32_t tiles_m, tiles_n;
    int32_t k_blocks;    // ceil(K / 128)
    int32_t out_fp32;
    int32_t accumulate;  // fp32 output: add to D
    uint32_t idesc;      // instruction descriptor without the scale-factor ids
    int32_t late;        // nothing here depends on the kernel before (sbl_b8_device.cuh)
    uint32_t *err;
};

// Scales move in groups of kB8SfBlocks K blocks (two words a row): every copy
// to tensor memory makes the MMAs behind it wait, and a copy of two words costs
// little more than one (without loads, 16384 x 2048 x 11008 took 245 us with one
// word a copy, 231 with two, 235 without any copy).  Two groups have room, in
// shared memory (where a slot is loaded) and in tensor memory next to the two
// accumulators of BN columns (4 columns for 128 A rows, 4 per 128 B rows, a word).
constexpr int kB8SfBlocks = 8;
constexpr int kB8SfBufs = 2;
// Epilogue staging: one block of 32 rows x 64 bytes per epilogue warp.
constexpr int kB8EpiBufBytes = 32 * 64;
constexpr int kB8EpiBytes = kEpiWarps * kB8EpiBufBytes;

// The most shared memory a CTA can have.
constexpr int kB8SmemAll = 227 * 1024;

template <int BN>
struct B8Cfg {
    static_assert(BN == 128 || BN == 256, "tile width");
    static constexpr int kBBytes = BN * kBKBytes;
    static constexpr int kSfaBytes = 512;
    static constexpr int kSfbBytes = BN * 4;
    static constexpr int kSfWordBytes = kSfaBytes + kSfbBytes;  // one word of every row
    static constexpr int kSfBytes = kB8SfBlocks / 4 * kSfWordBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;
    // six, or four of the 48 KiB ones; five instead of six measured the same
    static constexpr int kStages = (kB8SmemAll - 1024 - kB8EpiBytes - kB8SfBufs * kSfBytes - 256) / kStageBytes;
    static constexpr int kSfWordCols = 4 + BN / 32;
    static constexpr int kSfCols = kB8SfBlocks / 4 * kSfWordCols;
    static constexpr int kSfCol0 = kTmemCols - kB8SfBufs * kSfCols;
    // second accumulator: next to the first, or overlapping its last columns
    // where two do not fit beside the scales (see the epilogue)
    static constexpr int kAcc1 = 2 * BN <= kSfCol0 ? BN : (kSfCol0 - BN) / 32 * 32;
    static constexpr int kOverlap = BN - kAcc1;  // columns shared by the accumulators
    static_assert(kOverlap <= 64, "the first drained columns must free the overlap");
    static constexpr int kSmemBytes = kB8SmemAll;
};

// Instruction descriptor of kind::mxf8f6f4: B scale id (bits 4-5), A / B type
// (7-9, 10-12: 0 e4m3, 1 e5m2), N >> 3 (17-22), UE8M0 scales (23), M >> 4
// (24-28), A scale id (29-30).
__host__ __device__ constexpr uint32_t b8_idesc(int a_type, int b_type, int M, int N)
{
    return (static_cast<uint32_t>(a_type) << 7) | (static_cast<uint32_t>(b_type) << 10) |
           (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t b8_idesc_with_block(uint32_t idesc, int kb)
{
    const uint32_t id = static_cast<uint32_t>(kb & 3);
    return idesc | (id << 4) | (id << 29);
}

__device__ __forceinline__ void mma_b8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 512 bytes of scale words (128 rows x 4 blocks) to four columns of tensor
// memory, the same in each 32-lane quarter: 32 rows of 16 bytes, 8-row groups
// 128 bytes apart, no swizzle.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// Which stage last used each of the kB8SfBufs slots of a group ring: slots are
// taken in turn, so the oldest use is the next slot's.
struct SfUse {
    static_assert(kB8SfBufs == 2, "two slots");
    uint32_t groups = 0;             // groups so far
    uint32_t last[2] = {0u, 0u};     // 1 + stage of the slot's last use (0: none), oldest first
    __device__ __forceinline__ uint32_t slot() const { return groups & 1u; }
    __device__ __forceinline__ uint32_t oldest() const { return last[0] - 1u; }
    // the next slot was used fewer than `ring` stages before stage `now`
    __device__ __forceinline__ bool recent(uint32_t now, int ring) const
    {
        return last[0] != 0u && now - oldest() < static_cast<uint32_t>(ring);
    }
    __device__ __forceinline__ void use(uint32_t stage)
    {
        last[0] = last[1];
        last[1] = stage + 1u;
        ++groups;
    }
};

// D += block (fp32, element-wise in L2; each element of D gets one addition
// per launch, so the result does not depend on the order).
__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap *map, uint32_t src, int32_t c0, int32_t c1)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

// K blocks summed in tensor memory before the sum moves to registers (LONG).
constexpr int kB8SegBlocks = 32;
// K blocks of a bf16 result from which it is summed so as well.
constexpr int kB8MaxBf16Blocks = 512;

// LONG: results of long reductions, fp32 ones above all.  The tensor core truncates when it
// adds to its accumulator, so the error of a sum of n steps grows with n
// (relative to the result, measured on random operands: 1.0e-7 at K = 2048,
// 4.8e-7 at 8192, 1.2e-6 at 16384, where rounded additions give 1.9e-7).  The
// reduction is therefore cut into segments of kB8SegBlocks blocks, each
// summed in tensor memory and then added in registers with rounding.
//
// tmSA, tmSB: the scale words as [ceil(blocks / 4), padded rows] of 32 bits,
// boxes of 128 (A) and BN (B) words.
template <int BN, bool LONG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    b8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ CUtensorMap tmY, B8GemmArgs args)
{
    using Cfg = B8Cfg<BN>;
    constexpr int kStages = Cfg::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t a_base = base;
    const uint32_t b_base = a_base + kStages * kABytes;
    const uint32_t epi_base = b_base + kStages * Cfg::kBBytes;
    const uint32_t sf_base = epi_base + kB8EpiBytes;
    const uint32_t bar_base = sf_base + kB8SfBufs * Cfg::kSfBytes;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kStages + s); };
    auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * kStages + a); };
    auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * kStages + 2 + a); };
    const uint32_t drain_bar = bar_base + 8u * (2 * kStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (drain_bar + 8u - base));
    static_assert(8 * (2 * kStages + 6) <= 256, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_tiles = args.tiles_m * args.tiles_n;
    const int unit = static_cast<int>(blockIdx.x), units = static_cast<int>(gridDim.x);
    const int segments = LONG ? (args.k_blocks + kB8SegBlocks - 1) / kB8SegBlocks : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), kEpiWarps);  // one arrival per epilogue warp
        }
        mbar_init(drain_bar, 1);
        fence_barrier_init();
        tma_prefetch_map(&tmA);
        tma_prefetch_map(&tmB);
        tma_prefetch_map(&tmSA);
        tma_prefetch_map(&tmSB);
        tma_prefetch_map(&tmY);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (!args.late) grid_wait_and_release();

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t issued_mask = 0;
        uint32_t issued_phase[kStages];
        for (int s = 0; s < kStages; ++s) issued_phase[s] = 0;
        // Scales come with the first stage of their group.  A slot may be
        // filled again when the copy that read it, issued with the first stage
        // of group - kB8SfBufs, has finished: known from the ring if that
        // stage lies kStages back, else waited for.
        SfUse used;
        uint32_t count = 0;  // stages so far
        for (int tile = unit; ok && tile < num_tiles; tile += units) {
            int tm, tn;
            tile_coords(tile, args.tiles_m, args.tiles_n, tm, tn);
            const int arow = tm * kBM;
            const int brow = tn * BN;
            for (int kb = 0; kb < args.k_blocks; ++kb) {
                const bool ready = mbar_wait(empty_bar(stage), phase ^ 1u, args.err, kErrB8Gemm);
                if (!__all_sync(0xffffffffu, ready)) {
                    ok = false;
                    break;
                }
                const bool sf = kb % kB8SfBlocks == 0;
                if (sf) {
                    if (used.recent(count, kStages)) {
                        const uint32_t st = used.oldest();
                        const bool copied = mbar_wait(empty_bar(st % kStages), (st / kStages) & 1u, args.err, kErrB8Gemm);
                        if (!__all_sync(0xffffffffu, copied)) {
                            ok = false;
                            break;
                        }
                    }
                }
                if (lane == 0) {
                    const int words = sf ? min(kB8SfBlocks / 4, (args.k_blocks - kb + 3) >> 2) : 0;
                    const uint32_t bytes = Cfg::kStageBytes + words * Cfg::kSfWordBytes;
                    const uint32_t s = sf_base + used.slot() * Cfg::kSfBytes;
                    const uint32_t fb = full_bar(stage);
                    mbar_arrive_expect_tx(fb, bytes);
                    tma_load_2d(a_base + stage * kABytes, &tmA, kb * 128, arow, fb);
                    tma_load_2d(b_base + stage * Cfg::kBBytes, &tmB, kb * 128, brow, fb);
                    for (int w = 0; w < words; ++w) {
                        tma_load_2d(s + w * Cfg::kSfWordBytes, &tmSA, arow, (kb >> 2) + w, fb);
                        tma_load_2d(s + w * Cfg::kSfWordBytes + Cfg::kSfaBytes, &tmSB, tn * BN, (kb >> 2) + w, fb);
                    }
                }
                if (sf) used.use(count);
                ++count;
                __syncwarp();
                issued_mask |= 1u << stage;
                issued_phase[stage] = phase;
                if (++stage == kStages) stage = 0, phase ^= 1u;
            }
        }
        if (!ok) {
            // loads still in flight land before the CTA can exit
            for (int s = 0; s < kStages; ++s)
                if (issued_mask & (1u << s)) mbar_wait(full_bar(s), issued_phase[s], args.err, kErrB8Gemm);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        // Whole-warp control flow with one elected lane issuing: the
        // instructions want uniform registers, and what the compiler makes of a
        // lane-0 branch cost 5% (16384 x 2048 x 11008: 288 us against 269), the
        // same loop in one thread 14%.
        const bool elected = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int local = 0;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, args.err, kErrB8Gemm)) != 0;
        };
        // A buffer of scales may be written again when the MMAs that read it
        // have finished (the last stage of group - kB8SfBufs).
        SfUse read;
        uint32_t count = 0, sfa = 0;
        for (int tile = unit; ok && tile < num_tiles; tile += units) {
            for (int seg = 0; ok && seg < segments; ++seg, ++local) {
                const int kb0 = LONG ? seg * kB8SegBlocks : 0;
                const int kb1 = LONG ? min(kb0 + kB8SegBlocks, args.k_blocks) : args.k_blocks;
                const int acc = local & 1;
                // The accumulator's columns are free: with two disjoint ones
                // when tile local - 2 is drained; with overlapping ones when the
                // first columns of tile local - 1 are (all of local - 2 is by
                // then).
                if constexpr (Cfg::kOverlap > 0) {
                    if (local >= 1) ok = wait(tempty_bar(acc ^ 1), ((local - 1) >> 1) & 1);
                } else {
                    ok = wait(tempty_bar(acc), ((local >> 1) & 1) ^ 1);
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Cfg::kAcc1);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait(full_bar(stage), phase);
                    if (!ok) break;
                    const bool sf = kb % kB8SfBlocks == 0;
                    if (sf) {
                        if (read.recent(count, kStages)) {
                            const uint32_t st = read.oldest();
                            ok = wait(empty_bar(st % kStages), (st / kStages) & 1u);
                            if (!ok) break;
                        }
                        sfa = tmem_base + Cfg::kSfCol0 + read.slot() * Cfg::kSfCols;
                    }
                    tc_fence_after();
                    const uint32_t sft = sfa + ((kb % kB8SfBlocks) >> 2) * Cfg::kSfWordCols;
                    const uint32_t idesc = b8_idesc_with_block(args.idesc, kb);
                    const uint64_t adesc = smem_desc_k128(a_base + stage * kABytes);
                    const uint64_t bdesc = smem_desc_k128(b_base + stage * Cfg::kBBytes);
                    if (elected) {
                        if (sf) {
                            const uint32_t s = sf_base + read.slot() * Cfg::kSfBytes;
#pragma unroll
                            for (int w = 0; w < kB8SfBlocks / 4; ++w) {
                                if (kb + 4 * w >= args.k_blocks) break;
                                const uint32_t t = sfa + w * Cfg::kSfWordCols, sw = s + w * Cfg::kSfWordBytes;
                                tmem_cp_scales(t, sw);
#pragma unroll
                                for (int i = 0; i < BN / 128; ++i) tmem_cp_scales(t + 4 + 4 * i, sw + Cfg::kSfaBytes + 512 * i);
                            }
                        }
#pragma unroll
                        for (int kk = 0; kk < kBKBytes / 32; ++kk)
                            mma_b8(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, sft, sft + 4, (kb > kb0 || kk > 0) ? 1u : 0u);
                        // frees the stage (and the scales' slot) once these finish
                        tc_commit(empty_bar(stage));
                    }
                    __syncwarp();
                    // the group's last stage (of this tile) closes its buffer
                    if (kb % kB8SfBlocks == kB8SfBlocks - 1 || kb == args.k_blocks - 1) read.use(count);
                    ++count;
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                if (elected) {
                    tc_commit(tfull_bar(acc));
                }
                __syncwarp();
            }
        }
        // every MMA issued has completed before tensor memory is released
        if (elected) {
            tc_commit(drain_bar);
        }
        __syncwarp();
        mbar_wait(drain_bar, 0, args.err, kErrB8Gemm);
        __syncwarp();
    } else if (warp >= 2) {
        // ---------------------------------------------------- epilogue (warps 2-9)
        // Lane r of a warp drains TMEM row 32 (warp % 4) + r, 32 columns of
        // every 64 (warps 2-5 the first half).  With overlapping accumulators
        // the shared columns go first: the last 64 of the first accumulator,
        // the first 64 of the second, and the next tile's MMAs may start.
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const uint32_t buf = epi_base + static_cast<uint32_t>(warp - 2) * kB8EpiBufBytes;
        constexpr int kChunks = BN / 64;
        int local = 0;
        auto release = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(tempty_bar(acc));
            }
        };
        // one staged block: 32 rows of 64 bytes, 16-byte chunk c at
        // c ^ ((lane / 2) % 4) (64-byte swizzle), one TMA store
        auto store_block = [&](const uint32_t(&w)[16], int col, int row0) {
            if (lane == 0) bulk_wait_group_read<0>();  // the block before has left the buffer
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t addr = buf + static_cast<uint32_t>(lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16));
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[4 * c]), "r"(w[4 * c + 1]),
                             "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (args.accumulate)
                    tma_reduce_add_2d(&tmY, buf, col, row0);
                else
                    tma_store_2d(&tmY, buf, col, row0);
                bulk_commit_group();
            }
        };
        // 32 rows x 32 columns of this warp: one block in bf16, two in fp32
        auto store = [&](const uint32_t(&v)[32], int col, int row0) {
            if (col >= args.N || row0 >= args.M) return;  // warp-uniform: block outside D
            uint32_t w[16];
            if (!args.out_fp32) {
#pragma unroll
                for (int q = 0; q < 16; ++q) w[q] = pack_bf16(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
                store_block(w, col, row0);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (col + 16 * h >= args.N) break;
#pragma unroll
                    for (int q = 0; q < 16; ++q) w[q] = v[16 * h + q];
                    store_block(w, col + 16 * h, row0);
                }
            }
        };
        for (int tile = unit; tile < num_tiles; tile += units) {
            int tm, tn;
            tile_coords(tile, args.tiles_m, args.tiles_n, tm, tn);
            const int row0 = tm * kBM + quarter * 32;
            const int col0 = tn * BN + 32 * half;
            if constexpr (LONG) {
                float sum[kChunks][32];
#pragma unroll
                for (int j = 0; j < kChunks; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.0f;
                bool ready = true;
                for (int seg = 0; seg < segments; ++seg, ++local) {
                    const int acc = local & 1;
                    ready = __all_sync(0xffffffffu, mbar_wait(tfull_bar(acc), (local >> 1) & 1, args.err, kErrB8Gemm));
                    if (!ready) break;
                    tc_fence_after();
                    const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                           static_cast<uint32_t>(acc * Cfg::kAcc1 + 32 * half);
                    auto add = [&](int j, bool last) {
                        uint32_t v[32];
                        __syncwarp();
                        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(64 * j), v);
                        tmem_wait_ld();
                        if (last) release(acc);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[j][i] = __fadd_rn(sum[j][i], __uint_as_float(v[i]));
                    };
                    constexpr int kFree = Cfg::kOverlap > 0 ? 0 : kChunks - 1;
                    if (Cfg::kOverlap > 0 && acc == 0) {
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) add(kChunks - 1 - i, i == kFree);
                    } else {
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) add(i, i == kFree);
                    }
                }
                if (!ready) break;
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(sum[j][i]);
                    store(v, col0 + 64 * j, row0);
                }
            } else {
                const int acc = local & 1;
                const bool ready = mbar_wait(tfull_bar(acc), (local >> 1) & 1, args.err, kErrB8Gemm);
                if (!__all_sync(0xffffffffu, ready)) break;
                tc_fence_after();
                const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(acc * Cfg::kAcc1 + 32 * half);
#pragma unroll 1
                for (int i = 0; i < kChunks; ++i) {
                    const int j = (Cfg::kOverlap > 0 && acc == 0) ? kChunks - 1 - i : i;
                    uint32_t v[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(64 * j), v);
                    tmem_wait_ld();
                    if (i == (Cfg::kOverlap > 0 ? 0 : kChunks - 1)) release(acc);
                    store(v, col0 + 64 * j, row0);
                }
                ++local;
            }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
    if (args.late) grid_wait_and_release();
}

}  // namespace sbl
