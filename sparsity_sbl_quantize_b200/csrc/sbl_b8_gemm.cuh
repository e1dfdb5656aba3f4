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
// Tiles and roles are those of the other tcgen05 products: warp 0 TMA loads,
// warp 1 MMAs, warps 2-9 the epilogue.
#pragma once

#include <cuda_bf16.h>

#include "sbl_b8_format.cuh"
#include "sbl_device.cuh"
#include "sbl_gemm.cuh"  // tile raster, role sizes

namespace sbl {

struct B8GemmArgs {
    int32_t M, N;
    int32_t tiles_m, tiles_n;
    int32_t k_blocks;    // ceil(K / 128)
    int32_t out_fp32;
    int32_t accumulate;  // fp32 output: add to D
    uint32_t idesc;      // instruction descriptor without the scale-factor ids
    uint32_t *err;
};

// Columns of tensor memory: two accumulators of BN columns, then kB8SfBufs
// buffers of scale words (4 columns for 128 A rows, 4 per 128 B rows).  Four
// buffers in turn put 16 stages between two uses of a buffer, more than the
// ring holds, so a copy never meets MMAs that still read the old scales.
constexpr int kB8SfBufs = 4;

// A kernel that takes c of the 512 columns of tensor memory takes at least
// c / 512 of the SM's shared memory too (all of it here).  Then CTAs that fit
// on an SM together also find their tensor memory, whatever kernels and
// streams they belong to: an allocation that had to wait for another CTA,
// while both wait for cluster mates elsewhere, could close a circle.
constexpr int kB8SmemAll = 227 * 1024;

template <int BN, bool PAIR>
struct B8Cfg {
    static_assert(BN == 128 || BN == 256, "tile width");
    static constexpr int kBRows = PAIR ? BN / 2 : BN;
    static constexpr int kBBytes = kBRows * kBKBytes;
    static constexpr int kSfaBytes = 512;
    static constexpr int kSfbBytes = BN * 4;
    static constexpr int kSfBytes = kSfaBytes + kSfbBytes;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = (180 * 1024) / (kStageBytes + kSfBytes);
    static constexpr int kSfCols = 4 + BN / 32;
    static constexpr int kSfCol0 = kTmemCols - kB8SfBufs * kSfCols;
    // second accumulator: next to the first, or overlapping its last columns
    // where two do not fit beside the scales (see the epilogue)
    static constexpr int kAcc1 = 2 * BN <= kSfCol0 ? BN : (kSfCol0 - BN) / 32 * 32;
    static constexpr int kOverlap = BN - kAcc1;  // columns shared by the accumulators
    static_assert(kOverlap <= 64, "the first drained columns must free the overlap");
    static_assert(1024 + kStages * (kStageBytes + kSfBytes) + kEpiBytes + 256 <= kB8SmemAll, "shared memory");
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

template <bool PAIR>
__device__ __forceinline__ void mma_b8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa,
                                       uint32_t sfb, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
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
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(1u) << 16;
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

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

// LONG: fp32 results of long reductions.  The tensor core truncates when it
// adds to its accumulator, so the error of a sum of n steps grows with n
// (relative to the result, measured on random operands: 1.0e-7 at K = 2048,
// 4.8e-7 at 8192, 1.2e-6 at 16384, where rounded additions give 1.9e-7).  The
// reduction is therefore cut into segments of kB8SegBlocks blocks, each
// summed in tensor memory and then added in registers with rounding.
//
// tmSA, tmSB: the scale words as [ceil(blocks / 4), padded rows] of 32 bits,
// boxes of 128 (A) and BN (B) words: both CTAs of a pair need every B scale.
template <int BN, bool PAIR, bool LONG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    b8_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ CUtensorMap tmY, B8GemmArgs args)
{
    using Cfg = B8Cfg<BN, PAIR>;
    constexpr int kStages = Cfg::kStages;
    constexpr int kTileM = PAIR ? 2 * kBM : kBM;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    const uint32_t a_base = base;
    const uint32_t b_base = a_base + kStages * kABytes;
    const uint32_t epi_base = b_base + kStages * Cfg::kBBytes;
    const uint32_t sf_base = epi_base + kEpiBytes;
    const uint32_t bar_base = sf_base + kStages * Cfg::kSfBytes;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kStages + s); };
    auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * kStages + a); };
    auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * kStages + 2 + a); };
    const uint32_t drain_bar = bar_base + 8u * (2 * kStages + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (bar_base - base) + 224);
    static_assert(8 * (2 * kStages + 5) <= 224, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int num_tiles = args.tiles_m * args.tiles_n;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    const bool leader = rank == 0;
    const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int units = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
    const int segments = LONG ? (args.k_blocks + kB8SegBlocks - 1) / kB8SegBlocks : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), (PAIR ? 2 : 1) * kEpiWarps);  // one arrival per epilogue warp
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
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_addr(tmem_slot), kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_addr(tmem_slot), kTmemCols);
            tmem_relinquish();
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if constexpr (PAIR) cluster_sync_all();
    const uint32_t tmem_base = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        uint32_t issued_mask = 0;
        uint32_t issued_phase[kStages];
        for (int s = 0; s < kStages; ++s) issued_phase[s] = 0;
        for (int tile = unit; ok && tile < num_tiles; tile += units) {
            int tm, tn;
            tile_coords(tile, args.tiles_m, args.tiles_n, tm, tn);
            const int arow = tm * kTileM + static_cast<int>(rank) * kBM;
            const int brow = tn * BN + static_cast<int>(rank) * Cfg::kBRows;
            for (int kb = 0; kb < args.k_blocks; ++kb) {
                const bool ready = mbar_wait(empty_bar(stage), phase ^ 1u, args.err, kErrB8Gemm);
                if (!__all_sync(0xffffffffu, ready)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const bool sf = (kb & 3) == 0;  // this stage brings the scales of four
                    const uint32_t bytes = Cfg::kStageBytes + (sf ? Cfg::kSfBytes : 0);
                    const uint32_t sa = sf_base + stage * Cfg::kSfBytes, sb = sa + Cfg::kSfaBytes;
                    if constexpr (PAIR) {
                        const uint32_t fb = map_shared_rank(full_bar(stage), 0);
                        if (leader) mbar_arrive_expect_tx(full_bar(stage), 2 * bytes);
                        tma_load_2d_pair(a_base + stage * kABytes, &tmA, kb * 128, arow, fb);
                        tma_load_2d_pair(b_base + stage * Cfg::kBBytes, &tmB, kb * 128, brow, fb);
                        if (sf) {
                            tma_load_2d_pair(sa, &tmSA, arow, kb >> 2, fb);
                            tma_load_2d_pair(sb, &tmSB, tn * BN, kb >> 2, fb);
                        }
                    } else {
                        mbar_arrive_expect_tx(full_bar(stage), bytes);
                        tma_load_2d(a_base + stage * kABytes, &tmA, kb * 128, arow, full_bar(stage));
                        tma_load_2d(b_base + stage * Cfg::kBBytes, &tmB, kb * 128, brow, full_bar(stage));
                        if (sf) {
                            tma_load_2d(sa, &tmSA, arow, kb >> 2, full_bar(stage));
                            tma_load_2d(sb, &tmSB, tn * BN, kb >> 2, full_bar(stage));
                        }
                    }
                }
                __syncwarp();
                issued_mask |= 1u << stage;
                issued_phase[stage] = phase;
                if (++stage == kStages) stage = 0, phase ^= 1u;
            }
        }
        if (!ok && leader) {
            for (int s = 0; s < kStages; ++s)
                if (issued_mask & (1u << s)) mbar_wait(full_bar(s), issued_phase[s], args.err, kErrB8Gemm);
        }
    } else if (warp == 1 && leader) {
        // -------------------------------------------------------- MMA issuer
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        int local = 0;
        uint32_t sf_group = 0;  // groups of four stages so far
        for (int tile = unit; ok && tile < num_tiles; tile += units) {
            for (int seg = 0; ok && seg < segments; ++seg, ++local) {
                const int kb0 = LONG ? seg * kB8SegBlocks : 0;
                const int kb1 = LONG ? min(kb0 + kB8SegBlocks, args.k_blocks) : args.k_blocks;
                const int acc = local & 1;
                // The accumulator's columns are free: with two disjoint ones when
                // tile local - 2 is drained; with overlapping ones when the first
                // columns of tile local - 1 are (all of local - 2 is by then).
                bool free_acc = true;
                if constexpr (Cfg::kOverlap > 0) {
                    if (local >= 1)
                        free_acc = mbar_wait(tempty_bar(acc ^ 1), ((local - 1) >> 1) & 1, args.err, kErrB8Gemm);
                } else {
                    free_acc = mbar_wait(tempty_bar(acc), ((local >> 1) & 1) ^ 1, args.err, kErrB8Gemm);
                }
                if (!__all_sync(0xffffffffu, free_acc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * Cfg::kAcc1);
                uint32_t sfa = 0;
                for (int kb = kb0; kb < kb1; ++kb) {
                    const bool ready = mbar_wait(full_bar(stage), phase, args.err, kErrB8Gemm);
                    if (!__all_sync(0xffffffffu, ready)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if ((kb & 3) == 0) {
                        sfa = tmem_base + Cfg::kSfCol0 + (sf_group % kB8SfBufs) * Cfg::kSfCols;
                        ++sf_group;
                    }
                    if (lane == 0) {
                        if ((kb & 3) == 0) {
                            const uint32_t s = sf_base + stage * Cfg::kSfBytes;
                            tmem_cp_scales<PAIR>(sfa, s);
#pragma unroll
                            for (int i = 0; i < BN / 128; ++i)
                                tmem_cp_scales<PAIR>(sfa + 4 + 4 * i, s + Cfg::kSfaBytes + 512 * i);
                        }
                        const uint32_t idesc = b8_idesc_with_block(args.idesc, kb);
                        const uint64_t adesc = smem_desc_k128(a_base + stage * kABytes);
                        const uint64_t bdesc = smem_desc_k128(b_base + stage * Cfg::kBBytes);
#pragma unroll
                        for (int kk = 0; kk < kBKBytes / 32; ++kk)
                            mma_b8<PAIR>(d_tmem, adesc + 2 * kk, bdesc + 2 * kk, idesc, sfa, sfa + 4, (kb > kb0 || kk > 0) ? 1u : 0u);
                        if constexpr (PAIR)
                            tc_commit_pair(empty_bar(stage), 0x3);
                        else
                            tc_commit(empty_bar(stage));
                    }
                    __syncwarp();
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                if (lane == 0) {
                    if constexpr (PAIR)
                        tc_commit_pair(tfull_bar(acc), 0x3);
                    else
                        tc_commit(tfull_bar(acc));
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            if constexpr (PAIR)
                tc_commit_pair(drain_bar, 0x1);
            else
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
        const uint32_t buf = epi_base + static_cast<uint32_t>(warp - 2) * kEpiBufBytes;
        constexpr int kChunks = BN / 64;
        uint32_t nstore = 0;
        int local = 0;
        auto release = [&](int acc) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    mbar_arrive_cluster(map_shared_rank(tempty_bar(acc), 0));
                else
                    mbar_arrive(tempty_bar(acc));
            }
        };
        // 32 x 32 fp32 values of this warp to D (staged, swizzled, one TMA store)
        auto store = [&](const uint32_t(&v)[32], int col, int row0) {
            if (col >= args.N || row0 >= args.M) return;  // warp-uniform: block outside D
            if (!args.out_fp32) {
                // two 2 KiB staging halves in turn: rows of 64 bytes, chunk c
                // at c ^ ((lane / 2) % 4) (64-byte swizzle)
                const uint32_t sbuf = buf + static_cast<uint32_t>((nstore & 1) * (kEpiBufBytes / 2));
                if (lane == 0) bulk_wait_group_read<1>();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) w[q] = pack_bf16(__uint_as_float(v[8 * c + 2 * q]), __uint_as_float(v[8 * c + 2 * q + 1]));
                    const uint32_t addr = sbuf + static_cast<uint32_t>(lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16));
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                 : "memory");
                }
            } else {
                if (lane == 0) bulk_wait_group_read<0>();
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t addr = buf + static_cast<uint32_t>(lane * 128 + ((c ^ (lane & 7)) * 16));
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[4 * c]), "r"(v[4 * c + 1]),
                                 "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                                 : "memory");
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (!args.out_fp32)
                    tma_store_2d(&tmY, buf + static_cast<uint32_t>((nstore & 1) * (kEpiBufBytes / 2)), col, row0);
                else if (args.accumulate)
                    tma_reduce_add_2d(&tmY, buf, col, row0);
                else
                    tma_store_2d(&tmY, buf, col, row0);
                bulk_commit_group();
            }
            ++nstore;
        };
        for (int tile = unit; tile < num_tiles; tile += units) {
            int tm, tn;
            tile_coords(tile, args.tiles_m, args.tiles_n, tm, tn);
            const int row0 = tm * kTileM + static_cast<int>(rank) * kBM + quarter * 32;
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
    if constexpr (PAIR) cluster_sync_all();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem_base, kTmemCols);
        else
            tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace sbl
