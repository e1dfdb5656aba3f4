// sbl_b8_skinny.cuh -- the b8 product for few rows (tokens) on sm_100a.
//
//   Y[t, o] = sum_k x[t, k] W[o, k],   T <= 128
//
// With few tokens the product is one pass over W, so what counts is that every
// SM streams its share of W's bytes at once.  The operands swap places: 128
// rows of W are the MMA's M side (so no tensor-core row is spent on missing
// tokens) and the tokens, padded to NT, its N side; and K is split over the S
// CTAs of a cluster, so that few weight tiles still fill the device.  Each CTA
// sums its part of K in tensor memory; the parts meet in shared memory and
// every CTA adds 128 / S rows of them, in the order of the parts (the result
// does not depend on timing), reading its peers' shared memory.
//
// FUSED: X comes as bf16 and every CTA quantises the K range it needs itself
// (T x K / S values), writing codes and scales straight into the layouts the
// MMA reads; the clusters of the first weight tile also store them (the
// checkpoint).  This saves a launch, and costs each CTA T x K / S values of
// reading, so it is used while that is small.  Otherwise X is a b8 matrix and
// its blocks ride in the ring with W's.
#pragma once

#include <cuda_bf16.h>

#include "sbl_b8.cuh"
#include "sbl_b8_gemm.cuh"
#include "sbl_b8_device.cuh"

namespace sbl {

constexpr int kSkThreads = 512;
constexpr int kSkQuantWarps = 14;  // warps 2-15 quantise X
constexpr int kSkQuantBatch = 4;   // (token, block) pairs a half warp has in flight
constexpr int kSkMaxStages = 12;
constexpr int kSkMaxSplit = 8;     // the portable cluster size

struct SkinnyArgs {
    int32_t O, K, T;
    int32_t blocks;         // ceil(K / 128)
    int32_t split;          // CTAs of a cluster
    int32_t stages;
    int32_t max_groups;     // most scale words (of a row) in one CTA's K range
    int32_t max_blocks;     // most K blocks in one CTA's range
    uint32_t tmem_cols;
    uint32_t idesc;
    const uint16_t *X;      // FUSED: bf16 input
    int64_t ldx;
    uint8_t *xc;            // X's codes and scales: outputs (FUSED) or inputs
    int64_t ldc;
    uint32_t *xs;
    int64_t xrp;
    int32_t words;
    const uint32_t *ws;     // W's scales
    int64_t wrp;
    void *Y;
    int64_t ldy;
    int32_t y_fp32;
    int32_t accumulate;     // fp32 output: add to Y
    uint32_t *err;
};

// Bytes of a CTA's shared memory.  The ring is reused for the partial sums.
__host__ __device__ constexpr int64_t skinny_stage_bytes(int nt, bool fused) { return kABytes + (fused ? 0 : nt * kBKBytes); }

__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t cluster_addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

template <int TYPE, int NT, bool FUSED>
__global__ void __launch_bounds__(kSkThreads)
    b8_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, SkinnyArgs args)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    constexpr int kStageBytes = static_cast<int>(skinny_stage_bytes(NT, FUSED));
    const uint32_t x_base = base + args.stages * kStageBytes;  // FUSED: [blocks][NT][128] codes
    const uint32_t sfw_base = x_base + (FUSED ? args.max_blocks * NT * kBKBytes : 0);
    const uint32_t sfx_base = sfw_base + args.max_groups * 512;
    const uint32_t bar_base = sfx_base + args.max_groups * 512;
    auto full_bar = [&](int s) { return bar_base + 8u * s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (kSkMaxStages + s); };
    const uint32_t sf_bar = bar_base + 16u * kSkMaxStages;
    const uint32_t x_bar = sf_bar + 8u, done_bar = sf_bar + 16u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base_ptr + (sf_bar + 24u - base));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = args.split;
    const int tile = static_cast<int>(blockIdx.x) / S, rank = static_cast<int>(blockIdx.x) - tile * S;
    const int b0 = static_cast<int>(static_cast<int64_t>(rank) * args.blocks / S);
    const int b1 = static_cast<int>(static_cast<int64_t>(rank + 1) * args.blocks / S);
    const int g0 = b0 >> 2, groups = ((b1 - 1) >> 2) - g0 + 1;
    const int row0 = tile * kBM;

    if (threadIdx.x == 0) {
        for (int s = 0; s < args.stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(sf_bar, 1);
        mbar_init(x_bar, kSkQuantWarps);
        mbar_init(done_bar, 1);
        fence_barrier_init();
        tma_prefetch_map(&tmW);
        if constexpr (!FUSED) tma_prefetch_map(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(tmem_slot), args.tmem_cols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_wait_and_release();

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            const uint64_t pol = l2_evict_first_policy();
            mbar_arrive_expect_tx(sf_bar, static_cast<uint32_t>(groups) * (FUSED ? 512u : 1024u));
            for (int g = 0; g < groups; ++g) {
                bulk_load_1d(sfw_base + 512 * g, args.ws + (g0 + g) * args.wrp + row0, 512, sf_bar, pol);
                if constexpr (!FUSED) bulk_load_1d(sfx_base + 512 * g, args.xs + (g0 + g) * args.xrp, 512, sf_bar, pol);
            }
        }
        __syncwarp();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int b = b0; ok && b < b1; ++b) {
            ok = __all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, args.err, kErrB8Gemm));
            if (!ok) break;
            if (lane == 0) {
                const uint32_t s = base + stage * kStageBytes;
                mbar_arrive_expect_tx(full_bar(stage), kStageBytes);
                tma_load_2d(s, &tmW, b * 128, row0, full_bar(stage));
                if constexpr (!FUSED) tma_load_2d(s + kABytes, &tmX, b * 128, 0, full_bar(stage));
            }
            __syncwarp();
            if (++stage == args.stages) stage = 0, phase ^= 1u;
        }
        if (!ok) {
            // the loads in flight land before the CTA can exit: the stages
            // filled last, one phase each
            mbar_wait(sf_bar, 0, args.err, kErrB8Gemm);
            for (int s = 0; s < args.stages; ++s) mbar_wait(full_bar(s), s < stage ? phase : phase ^ 1u, args.err, kErrB8Gemm);
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        const bool elected = elect_one();
        const uint32_t sf_tmem = tmem_base + NT;
        bool ok = mbar_wait_spin(sf_bar, 0, args.err, kErrB8Gemm);
        if (FUSED && ok) ok = mbar_wait_spin(x_bar, 0, args.err, kErrB8Gemm);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok && elected)
            for (int g = 0; g < groups; ++g) {
                tmem_cp_scales(sf_tmem + 8 * g, sfw_base + 512 * g);
                tmem_cp_scales(sf_tmem + 8 * g + 4, sfx_base + 512 * g);
            }
        __syncwarp();
        int stage = 0;
        uint32_t phase = 0;
        for (int b = b0; ok && b < b1; ++b) {
            ok = __all_sync(0xffffffffu, mbar_wait_spin(full_bar(stage), phase, args.err, kErrB8Gemm));
            if (!ok) break;
            tc_fence_after();
            if (elected) {
                const uint32_t s = base + stage * kStageBytes;
                const uint32_t sf = sf_tmem + 8 * ((b >> 2) - g0);
                const uint32_t idesc = b8_idesc_with_block(args.idesc, b);
                const uint64_t wdesc = smem_desc_k128(s);
                const uint64_t xdesc = smem_desc_k128(FUSED ? x_base + (b - b0) * NT * kBKBytes : s + kABytes);
#pragma unroll
                for (int kk = 0; kk < kBKBytes / 32; ++kk)
                    mma_b8(tmem_base, wdesc + 2 * kk, xdesc + 2 * kk, idesc, sf, sf + 4, (b > b0 || kk > 0) ? 1u : 0u);
                tc_commit(empty_bar(stage));
            }
            __syncwarp();
            if (++stage == args.stages) stage = 0, phase ^= 1u;
        }
        // every MMA issued has completed: the epilogue's signal, and before
        // tensor memory is released
        if (elected) tc_commit(done_bar);
        __syncwarp();
    } else if constexpr (FUSED) {
        // ------------------------------------ quantise X's part (warps 2-15)
        // a half warp per (token, block), kBatch at a time to have the loads in
        // flight together
        constexpr int kHalves = 2 * kSkQuantWarps, kBatch = kSkQuantBatch;
        const int hw = 2 * (warp - 2) + (lane >> 4), l = lane & 15;
        const int nb = b1 - b0, items = args.T * nb;
        uint8_t *sfx = base_ptr + (sfx_base - base);
        for (int first = 0; first < items; first += kBatch * kHalves) {
            uint4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (first + j * kHalves >= items) break;
                const int item = first + j * kHalves + hw;
                const int t = item / nb, b = b0 + item - t * nb;
                const int64_t c = static_cast<int64_t>(b) * 128 + 8 * l;
                v[j] = item < items && c < args.K ? __ldg(reinterpret_cast<const uint4 *>(args.X + t * args.ldx + c))
                                                  : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (first + j * kHalves >= items) break;
                const int item = first + j * kHalves + hw;
                const int t = item / nb, b = b0 + item - t * nb;
                const uint32_t byte = b8_scale_byte<TYPE>(half_warp_max(bf16x8_absmax(v[j])) << 16);
                const uint2 q = b8_encode_bf16x8<TYPE>(v[j], b8_inv_scale(byte));
                if (item >= items) continue;
                const uint32_t addr = x_base + (b - b0) * NT * kBKBytes + t * 128 + (((l >> 1) ^ (t & 7)) << 4) + 8 * (l & 1);
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(q.x), "r"(q.y) : "memory");
                const int64_t c = static_cast<int64_t>(b) * 128 + 8 * l;
                if (l == 0) sfx[512 * ((b >> 2) - g0) + 4 * (4 * (t & 31) + (t >> 5)) + (b & 3)] = static_cast<uint8_t>(byte);
                if (tile == 0) {
                    if (c < args.K) *reinterpret_cast<uint2 *>(args.xc + t * args.ldc + c) = q;
                    if (l == 0)
                        reinterpret_cast<uint8_t *>(args.xs + b8_word_index(b >> 2, args.xrp, t))[b & 3] = static_cast<uint8_t>(byte);
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(x_bar);
        if (tile == 0 && rank == 0) {
            // the checkpoint's padding: whole words of padded rows, bytes of
            // padded blocks
            const int i0 = threadIdx.x - 64;
            const int rows = static_cast<int>(args.xrp);
            for (int i = i0; i < rows * args.words; i += 32 * kSkQuantWarps) {
                const int w = i / rows, t = i - w * rows;
                if (t >= args.T)
                    args.xs[b8_word_index(w, args.xrp, t)] = kB8PadWord;
                else if (w == args.words - 1)
                    for (int b = args.blocks; b < 4 * args.words; ++b)
                        reinterpret_cast<uint8_t *>(args.xs + b8_word_index(w, args.xrp, t))[b & 3] = 127;
            }
        }
    }

    // -------------------------------------------- partial sums to shared memory
    // warps 2-5 own the four 32-lane quarters of tensor memory; the ring is
    // free once every MMA is done
    const bool done = mbar_wait(done_bar, 0, args.err, kErrB8Gemm);
    const bool all_done = __all_sync(0xffffffffu, done);
    tc_fence_after();
    float *part = reinterpret_cast<float *>(base_ptr);  // [T][128]
    if (warp >= 2 && warp < 6 && all_done) {
        const int quarter = warp & 3;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < NT && c < args.T; c += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_row + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < args.T) part[(c + j) * 128 + quarter * 32 + lane] = __uint_as_float(v[j]);
        }
        tc_fence_before();
    }
    __syncthreads();
    // Tensor memory goes back before this CTA waits for its peers: no CTA ever
    // holds some while it waits for another one, whose allocation might be
    // waiting for it.
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, args.tmem_cols);
    }
    if (S > 1) cluster_sync_all();
    // this CTA's rows [r0, r0 + 128 / S) of every token, four rows a thread,
    // every part's load in flight before the first is added
    const int quads = kBM / 4 / S, r0 = rank * (kBM / S);
    for (int i = threadIdx.x; i < args.T * quads; i += kSkThreads) {
        const int t = i / quads, r = r0 + 4 * (i - t * quads);
        const uint32_t at = base + 4u * (t * 128 + r);
        float4 v[kSkMaxSplit];
#pragma unroll
        for (int p = 0; p < kSkMaxSplit; ++p)
            if (p < S) v[p] = ld_shared_cluster_v4(S > 1 ? map_shared_rank(at, p) : at);
        float4 y = v[0];
#pragma unroll
        for (int p = 1; p < kSkMaxSplit; ++p)
            if (p < S) y.x += v[p].x, y.y += v[p].y, y.z += v[p].z, y.w += v[p].w;
        const int o = row0 + r;
        if (o >= args.O) continue;  // O is a multiple of 16
        if (args.y_fp32) {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(args.Y) + t * args.ldy + o);
            if (args.accumulate) {
                const float4 c = *d;
                y.x += c.x, y.y += c.y, y.z += c.z, y.w += c.w;
            }
            *d = y;
        } else {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(args.Y) + t * args.ldy + o) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        }
    }
    if (S > 1) cluster_sync_all();  // no CTA leaves while a peer reads its sums
}

}  // namespace sbl
