// sbl_b8_api.cu -- host side of the 8-bit block operators declared in
// include/sbl.h: argument validation, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <mutex>

#include "sbl.h"
#include "sbl_act_norm.cuh"
#include "sbl_b8.cuh"
#include "sbl_b8_gemm.cuh"
#include "sbl_b8_skinny.cuh"
#include "sbl_ckpt.cuh"
#include "sbl_host.h"

namespace sbl {

// Rows of a b8 matrix: tile coordinates and their products stay in 32 bits.
constexpr int64_t kB8MaxRows = 1ll << 30;

static std::mutex g_b8_mutex;
static bool g_b8_ready[kMaxDevices];

static bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// host_device, and once per device the shared-memory limits of this file's kernels.
static sbl_status b8_device(HostDevice *hd)
{
    const sbl_status st = host_device(hd);
    if (st != SBL_OK) return st;
    std::lock_guard<std::mutex> lock(g_b8_mutex);
    if (!g_b8_ready[hd->index]) {
        sbl_status st2 = SBL_OK;
        auto allow = [&](auto kernel) {
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kB8SmemAll) != cudaSuccess) st2 = SBL_ERR_CUDA;
        };
        allow(b8_gemm_kernel<128, false>);
        allow(b8_gemm_kernel<128, true>);
        allow(b8_gemm_kernel<256, false>);
        allow(b8_gemm_kernel<256, true>);
        allow(b8_skinny_kernel<kB8E4M3, 16, true>);
        allow(b8_skinny_kernel<kB8E4M3, 32, true>);
        allow(b8_skinny_kernel<kB8E4M3, 64, true>);
        allow(b8_skinny_kernel<kB8E5M2, 16, true>);
        allow(b8_skinny_kernel<kB8E5M2, 32, true>);
        allow(b8_skinny_kernel<kB8E5M2, 64, true>);
        allow(b8_skinny_kernel<0, 16, false>);
        allow(b8_skinny_kernel<0, 32, false>);
        allow(b8_skinny_kernel<0, 64, false>);
        allow(b8_skinny_kernel<0, 128, false>);
        if (st2 != SBL_OK) {
            cudaGetLastError();
            return st2;
        }
        g_b8_ready[hd->index] = true;
    }
    return SBL_OK;
}

// The status of a launch or a memset.  A failed one (a stream whose capture was broken, say)
// leaves no error behind: it would be taken for the next call's.
static sbl_status launched(cudaError_t e)
{
    if (e == cudaSuccess) return SBL_OK;
    cudaGetLastError();
    return SBL_ERR_CUDA;
}

// Launch with programmatic dependent launch: a kernel waits for the one before
// it (griddepcontrol.wait) before it touches global memory, or, one that neither
// reads nor writes what the one before it writes (`late`), before it ends.
template <typename... P, typename... A>
static sbl_status launch2(void (*kernel)(P...), int64_t grid, int64_t grid_y, int block, size_t smem, cudaStream_t stream, A... args)
{
    if (grid > 0x7fffffffll || grid_y > 65535) return SBL_ERR_SHAPE;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(grid_y));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

template <typename... P, typename... A>
static sbl_status launch(void (*kernel)(P...), int64_t grid, int block, size_t smem, cudaStream_t stream, A... args)
{
    return launch2(kernel, grid, 1, block, smem, stream, args...);
}

// The same in clusters of `cluster` CTAs.
template <typename... P, typename... A>
static sbl_status launch_cluster(void (*kernel)(P...), int64_t grid, int cluster, int block, cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Scale words (512 columns) a warp of the element-wise kernels takes: one
// while the rows alone do not fill the device twice over, four after that.
static int32_t words_per_warp(int64_t rows, int32_t words, int num_sms)
{
    const int64_t fit = rows * words / (2 * 64ll * num_sms);
    return static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({4, fit, words})));
}

template <typename Args>
static sbl_status launch_walk(const HostDevice &hd, void (*kernel)(Args), int64_t rows, Args a, cudaStream_t stream)
{
    // many long rows: a CTA a row (gated backward of 16384 x 11008 from e4m3 checkpoints 231 -> 214 us)
    if (a.words >= 8 && rows >= 8ll * hd.num_sms) {
        a.per_warp = 0;
        return launch2(kernel, rows, 1, 256, 0, stream, a);
    }
    a.per_warp = words_per_warp(rows, a.words, hd.num_sms);
    return launch2(kernel, (rows + 7) / 8, (a.words + a.per_warp - 1) / a.per_warp, 256, 0, stream, a);
}

// ------------------------------------------------------------ descriptors --
static sbl_status check_b8(const sbl_b8_desc *d)
{
    if (!d) return SBL_ERR_INVALID_ARG;
    if (d->type != SBL_B8_E4M3 && d->type != SBL_B8_E5M2 && d->type != SBL_B8_I8) return SBL_ERR_INVALID_ARG;
    if (d->rows < 0 || d->rows > kB8MaxRows || d->cols < 1 || d->cols > kB8MaxRows) return SBL_ERR_SHAPE;
    return SBL_OK;
}

// Matrices read or written by the element-wise kernels: rows of whole 16-byte
// pieces, as every activation of the library.
static sbl_status check_b8_act(const sbl_b8_desc *d)
{
    const sbl_status st = check_b8(d);
    if (st != SBL_OK) return st;
    if (d->cols < 16 || d->cols % 16 != 0 || d->cols > kMaxDim) return SBL_ERR_SHAPE;
    return SBL_OK;
}

static int64_t b8_ld(const sbl_b8_desc *d) { return round_up(d->cols, 16); }
static int64_t b8_rp(int64_t rows) { return round_up(rows, 128); }
static int32_t b8_words(int64_t cols) { return static_cast<int32_t>((cols + 511) / 512); }
static int64_t b8_scale_size(const sbl_b8_desc *d) { return 4 * b8_rp(d->rows) * b8_words(d->cols); }

static bool complete(const sbl_b8 *m) { return m && m->codes && m->scales; }
static bool b8_aligned(const sbl_b8 *m) { return aligned16(m->codes) && aligned16(m->scales); }
static uint32_t *scale_words(const sbl_b8 *m) { return reinterpret_cast<uint32_t *>(m->scales); }

// Whether every row of a strided bf16 matrix is 32-byte aligned (nullptr: yes).
static bool rows32(const void *p, int64_t ld) { return !p || ((reinterpret_cast<uintptr_t>(p) & 31u) == 0 && ld % 16 == 0); }

// A strided bf16 (or fp32) matrix of `cols` columns: 16-byte aligned rows.
static sbl_status check_strided(const void *p, int64_t ld, int64_t cols, int elem_bytes)
{
    if (ld < cols || ld > (1ll << 40) || (ld * elem_bytes) % 16 != 0) return SBL_ERR_SHAPE;
    return aligned16(p) ? SBL_OK : SBL_ERR_ALIGNMENT;
}

// -------------------------------------------------------------- quantiser --
template <int TYPE, int SRC>
static sbl_status quantize_rows(const HostDevice &hd, const sbl_b8_desc *d, const void *X, int64_t ldx, const sbl_b8 *out, cudaStream_t stream)
{
    B8RowArgs a;
    memset(&a, 0, sizeof(a));
    a.X = X;
    a.ldx = ldx;
    a.rows = d->rows;
    a.cols = d->cols;
    a.codes = out->codes;
    a.ldc = b8_ld(d);
    a.scales = scale_words(out);
    a.rp = b8_rp(d->rows);
    a.words = b8_words(d->cols);
    a.v32 = rows32(X, ldx);
    return launch_walk(hd, b8_quantize_rows_kernel<TYPE, SRC>, a.rp, a, stream);
}

template <int TYPE, int SRC, int SRC_TYPE, bool TILES>
static sbl_status quantize_tiles(const sbl_b8_desc *d, const void *X, int64_t ldx, const uint32_t *xs, const sbl_b8 *out,
                                 const sbl_b8 *out_t, cudaStream_t stream, bool late = false)
{
    B8TileArgs a;
    memset(&a, 0, sizeof(a));
    a.late = late ? 1 : 0;
    a.X = X;
    a.ldx = ldx;
    a.xs = xs;
    a.xrp = b8_rp(d->rows);
    a.rows = d->rows;
    a.cols = d->cols;
    if (out) {
        a.codes = out->codes;
        a.ldc = b8_ld(d);
        a.scales = scale_words(out);
        a.rp = b8_rp(d->rows);
    }
    if (out_t) {
        a.codes_t = out_t->codes;
        a.ldt = round_up(d->rows, 16);
        a.scales_t = scale_words(out_t);
        a.rpt = b8_rp(d->cols);
    }
    a.tiles_c = (d->cols + 127) / 128;
    return launch(b8_tile_kernel<TYPE, SRC, SRC_TYPE, TILES>, b8_rp(d->rows) / 128 * a.tiles_c, 256, 0, stream, a);
}

template <int TYPE>
static sbl_status quantize_type(const HostDevice &hd, const sbl_b8_desc *d, const void *X, bool fp32, int64_t ldx, bool tiles, const sbl_b8 *out,
                                const sbl_b8 *out_t, cudaStream_t stream)
{
    if (!tiles && !out_t)
        return fp32 ? quantize_rows<TYPE, kSrcF32>(hd, d, X, ldx, out, stream) : quantize_rows<TYPE, kSrcBf16>(hd, d, X, ldx, out, stream);
    if (tiles)
        return fp32 ? quantize_tiles<TYPE, kSrcF32, 0, true>(d, X, ldx, nullptr, out, out_t, stream)
                    : quantize_tiles<TYPE, kSrcBf16, 0, true>(d, X, ldx, nullptr, out, out_t, stream);
    return fp32 ? quantize_tiles<TYPE, kSrcF32, 0, false>(d, X, ldx, nullptr, out, out_t, stream)
                : quantize_tiles<TYPE, kSrcBf16, 0, false>(d, X, ldx, nullptr, out, out_t, stream);
}

static sbl_status quantize(const HostDevice &hd, const sbl_b8_desc *d, const void *X, bool fp32, int64_t ldx, bool tiles, const sbl_b8 *out,
                           const sbl_b8 *out_t, cudaStream_t stream)
{
    switch (d->type) {
    case SBL_B8_E4M3: return quantize_type<kB8E4M3>(hd, d, X, fp32, ldx, tiles, out, out_t, stream);
    case SBL_B8_E5M2: return quantize_type<kB8E5M2>(hd, d, X, fp32, ldx, tiles, out, out_t, stream);
    default: return quantize_type<kB8I8>(hd, d, X, fp32, ldx, tiles, out, out_t, stream);
    }
}

template <int SRC_TYPE>
static sbl_status transpose_from(const sbl_b8_desc *d, const sbl_b8 *in, int32_t type_t, const sbl_b8 *out_t, bool late, cudaStream_t stream)
{
    const int64_t ld = b8_ld(d);
    switch (type_t) {
    case SBL_B8_E4M3: return quantize_tiles<kB8E4M3, kSrcB8, SRC_TYPE, false>(d, in->codes, ld, scale_words(in), nullptr, out_t, stream, late);
    case SBL_B8_E5M2: return quantize_tiles<kB8E5M2, kSrcB8, SRC_TYPE, false>(d, in->codes, ld, scale_words(in), nullptr, out_t, stream, late);
    default: return quantize_tiles<kB8I8, kSrcB8, SRC_TYPE, false>(d, in->codes, ld, scale_words(in), nullptr, out_t, stream, late);
    }
}

// late: the kernel enqueued before writes nothing that this one reads or writes
static sbl_status transpose(const sbl_b8_desc *d, const sbl_b8 *in, int32_t type_t, const sbl_b8 *out_t, bool late, cudaStream_t stream)
{
    switch (d->type) {
    case SBL_B8_E4M3: return transpose_from<kB8E4M3>(d, in, type_t, out_t, late, stream);
    case SBL_B8_E5M2: return transpose_from<kB8E5M2>(d, in, type_t, out_t, late, stream);
    default: return transpose_from<kB8I8>(d, in, type_t, out_t, late, stream);
    }
}

// ----------------------------------------------------------------- product --
static bool encode_2d(const HostDevice &hd, CUtensorMap *map, CUtensorMapDataType dt, const void *base,
                      int64_t inner, int64_t rows, int64_t stride_bytes, int box_inner, int box_rows, CUtensorMapSwizzle sw,
                      CUtensorMapL2promotion promo)
{
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_bytes)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return hd.encode(map, dt, 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, promo,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool encode_codes(const HostDevice &hd, CUtensorMap *map, const sbl_b8_desc *d, const sbl_b8 *m, int box_rows)
{
    return encode_2d(hd, map, CU_TENSOR_MAP_DATA_TYPE_UINT8, m->codes, d->cols, d->rows, b8_ld(d), kBKBytes, box_rows,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

static bool encode_scales(const HostDevice &hd, CUtensorMap *map, const sbl_b8_desc *d, const sbl_b8 *m, int box_words)
{
    const int64_t rp = b8_rp(d->rows);
    return encode_2d(hd, map, CU_TENSOR_MAP_DATA_TYPE_UINT32, m->scales, rp, b8_words(d->cols), rp * 4, box_words, 1,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int BN, bool LONG>
static sbl_status launch_b8_gemm(const HostDevice &hd, const sbl_b8_desc *ad, const sbl_b8 *A, const sbl_b8_desc *bd, const sbl_b8 *B,
                                 void *D, int64_t ldd, B8GemmArgs args, cudaStream_t stream)
{
    using Cfg = B8Cfg<BN>;
    CUtensorMap ta, tb, tsa, tsb, ty;
    const bool fp32 = args.out_fp32 != 0;
    if (!encode_codes(hd, &ta, ad, A, kBM) || !encode_codes(hd, &tb, bd, B, BN) ||
        !encode_scales(hd, &tsa, ad, A, kBM) || !encode_scales(hd, &tsb, bd, B, BN) ||
        !encode_2d(hd, &ty, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, D, args.N,
                   args.M, ldd * (fp32 ? 4 : 2), fp32 ? 16 : 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE))
        return SBL_ERR_CUDA;
    args.tiles_m = static_cast<int32_t>((static_cast<int64_t>(args.M) + kBM - 1) / kBM);
    args.tiles_n = (args.N + BN - 1) / BN;
    const int64_t tiles = static_cast<int64_t>(args.tiles_m) * args.tiles_n;
    // 32-bit tile numbers and, per CTA, stage counts
    if (tiles > 0x3fffffff || (tiles / hd.num_sms + 1) * args.k_blocks > 0x7fffffff) return SBL_ERR_SHAPE;
    args.idesc = b8_idesc(ad->type, bd->type, kBM, BN);
    args.err = hd.err;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, hd.num_sms)));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, b8_gemm_kernel<BN, LONG>, ta, tb, tsa, tsb, ty, args));
}

// How the product of few tokens runs: padded tokens, CTAs that share K, stages.
struct SkinnyPlan {
    int nt, split, stages, max_blocks, max_groups, tmem_cols;
    int64_t smem;
};

static SkinnyPlan skinny_plan(int num_sms, int32_t O, int32_t K, int32_t T, bool fused)
{
    SkinnyPlan p;
    p.nt = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
    const int64_t tiles = (O + kBM - 1) / kBM;
    const int blocks = (K + 127) / 128;
    // Enough CTAs for every SM, two blocks each at least.  More of them
    // measured slower (6912 x 2560: 216 CTAs 7.1 us, 432 11.3).
    p.split = 1;
    while (p.split < kSkMaxSplit && tiles * p.split < num_sms && blocks >= 4 * p.split) p.split *= 2;
    p.max_blocks = (blocks + p.split - 1) / p.split;
    p.max_groups = (p.max_blocks + 2) / 4 + 1;
    // As many stages as fit when the CTAs of one round share the SMs, two to
    // an SM at least: at one to an SM the clusters of eight do not all find
    // room at once (2048 x 11008: 15.1 us instead of 7.9).
    const int64_t ctas = std::min<int64_t>(std::max<int64_t>((tiles * p.split + num_sms - 1) / num_sms, 2), 4);
    const int64_t fixed = 1024 + (fused ? static_cast<int64_t>(p.max_blocks) * p.nt * kBKBytes : 0) + 1024ll * p.max_groups + 512;
    const int64_t room = (kB8SmemAll - 1024 * ctas) / ctas - fixed;
    p.stages = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>({p.max_blocks, room / skinny_stage_bytes(p.nt, fused), kSkMaxStages})));
    p.tmem_cols = 32;
    while (p.tmem_cols < p.nt + 8 * p.max_groups) p.tmem_cols *= 2;
    p.smem = fixed + p.stages * skinny_stage_bytes(p.nt, fused);
    return p;
}

template <int TYPE, int NT, bool FUSED>
static sbl_status launch_skinny_nt(const HostDevice &hd, const SkinnyPlan &p, const sbl_b8_desc *wd, const sbl_b8 *W, const sbl_b8_desc *xd,
                                   const sbl_b8 *xq, SkinnyArgs a, cudaStream_t stream)
{
    CUtensorMap tw, tx;
    memset(&tx, 0, sizeof(tx));
    if (!encode_codes(hd, &tw, wd, W, kBM) || (!FUSED && !encode_codes(hd, &tx, xd, xq, NT))) return SBL_ERR_CUDA;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>((wd->rows + kBM - 1) / kBM * p.split));
    cfg.blockDim = dim3(kSkThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return launched(cudaLaunchKernelEx(&cfg, b8_skinny_kernel<TYPE, NT, FUSED>, tw, tx, a));
}

// Y [T, O] = X W^T for few tokens.  X: bf16 (quantised in the kernel, xq an
// output) or nullptr (xq an input).
static sbl_status skinny(const HostDevice &hd, const SkinnyPlan &p, const sbl_b8_desc *wd, const sbl_b8 *W, const sbl_b8_desc *xd,
                         const uint16_t *X, int64_t ldx, const sbl_b8 *xq, void *Y, int64_t ldy, bool fp32, bool accumulate, cudaStream_t stream)
{
    SkinnyArgs a;
    memset(&a, 0, sizeof(a));
    a.O = wd->rows;
    a.K = wd->cols;
    a.T = xd->rows;
    a.blocks = (a.K + 127) / 128;
    a.split = p.split;
    a.stages = p.stages;
    a.max_groups = p.max_groups;
    a.max_blocks = p.max_blocks;
    a.tmem_cols = static_cast<uint32_t>(p.tmem_cols);
    a.idesc = b8_idesc(wd->type, xd->type, kBM, p.nt);
    a.X = X;
    a.ldx = ldx;
    a.xc = xq->codes;
    a.ldc = b8_ld(xd);
    a.xs = scale_words(xq);
    a.xrp = b8_rp(xd->rows);
    a.words = b8_words(xd->cols);
    a.ws = scale_words(W);
    a.wrp = b8_rp(wd->rows);
    a.Y = Y;
    a.ldy = ldy;
    a.y_fp32 = fp32 ? 1 : 0;
    a.accumulate = accumulate ? 1 : 0;
    a.err = hd.err;
    const bool e5 = xd->type == SBL_B8_E5M2;
    if (!X) {
        switch (p.nt) {
        case 16: return launch_skinny_nt<0, 16, false>(hd, p, wd, W, xd, xq, a, stream);
        case 32: return launch_skinny_nt<0, 32, false>(hd, p, wd, W, xd, xq, a, stream);
        case 64: return launch_skinny_nt<0, 64, false>(hd, p, wd, W, xd, xq, a, stream);
        default: return launch_skinny_nt<0, 128, false>(hd, p, wd, W, xd, xq, a, stream);
        }
    }
    switch (p.nt) {
    case 16:
        return e5 ? launch_skinny_nt<kB8E5M2, 16, true>(hd, p, wd, W, xd, xq, a, stream)
                  : launch_skinny_nt<kB8E4M3, 16, true>(hd, p, wd, W, xd, xq, a, stream);
    case 32:
        return e5 ? launch_skinny_nt<kB8E5M2, 32, true>(hd, p, wd, W, xd, xq, a, stream)
                  : launch_skinny_nt<kB8E4M3, 32, true>(hd, p, wd, W, xd, xq, a, stream);
    default:
        return e5 ? launch_skinny_nt<kB8E5M2, 64, true>(hd, p, wd, W, xd, xq, a, stream)
                  : launch_skinny_nt<kB8E4M3, 64, true>(hd, p, wd, W, xd, xq, a, stream);
    }
}

// D = A B^T; every argument checked.  late: the kernel enqueued before writes
// neither operand and does not touch D.
static sbl_status gemm(const HostDevice &hd, const sbl_b8_desc *ad, const sbl_b8 *A, const sbl_b8_desc *bd, const sbl_b8 *B, void *D,
                       int64_t ldd, bool fp32, bool accumulate, bool late, cudaStream_t stream)
{
    B8GemmArgs args;
    memset(&args, 0, sizeof(args));
    args.late = late ? 1 : 0;
    args.M = ad->rows;
    args.N = bd->rows;
    args.k_blocks = (ad->cols + 127) / 128;
    args.out_fp32 = fp32 ? 1 : 0;
    args.accumulate = accumulate ? 1 : 0;
    // Few rows: the kernel that splits K.  It measured faster up to 64 rows
    // (n x k: 6912 x 2560 at 64: 9.1 us against 11.0; 2560 x 6912: 9.5 against 23.5),
    // and to 128 only where the other's tiles leave most SMs idle (2560 x 6912 at
    // 128: 11.6 against 23.8; 11008 x 2048: 13.4 against 10.4).
    const int64_t tiles_w = (args.N + kBM - 1) / kBM;
    if (args.M <= 64 || (args.M <= 128 && 4 * tiles_w <= hd.num_sms)) {
        const SkinnyPlan p = skinny_plan(hd.num_sms, bd->rows, bd->cols, ad->rows, false);
        // not for fp32 sums that need LONG, nor for a K whose scales do not fit
        if ((!fp32 || p.max_blocks <= kB8SegBlocks) && p.smem <= kB8SmemAll && p.tmem_cols <= kTmemCols)
            return skinny(hd, p, bd, B, ad, nullptr, 0, A, D, ldd, fp32, accumulate, stream);
    }
    // 128 x 256 tiles or 128 x 128 ones, of which a product with few tiles has
    // twice as many: the time of a launch in units of 10 ns fits
    // 460 + rounds (42 blocks + 60) and 340 + rounds (34 blocks + 45)
    // (m x n x k: 16384 x 2048 x 11008: 269 against 440 us; 512 x 6912 x 2560: 14.0 against 18.3;
    // 300 x 4864 x 896: 6.6 against 5.9; 777 x 1536 x 1536: 8.5 against 8.0).
    auto rounds = [&](int64_t bn) {
        return ((static_cast<int64_t>(args.M) + kBM - 1) / kBM * ((args.N + bn - 1) / bn) + hd.num_sms - 1) / hd.num_sms;
    };
    const bool wide = 460 + rounds(256) * (42ll * args.k_blocks + 60) <= 340 + rounds(128) * (34ll * args.k_blocks + 45);
    // bf16 results of a very long K are summed in segments too: over products of
    // one sign the tensor core's truncation reaches 2^-23 of the sum every 32 of K,
    // at 65536 a sixteenth of the half step (600000: off by one step in places),
    // and one accumulator over all of K would outlast the epilogue's wait
    const bool lng = args.k_blocks > (fp32 ? kB8SegBlocks : kB8MaxBf16Blocks);
    if (wide)
        return lng ? launch_b8_gemm<256, true>(hd, ad, A, bd, B, D, ldd, args, stream)
                   : launch_b8_gemm<256, false>(hd, ad, A, bd, B, D, ldd, args, stream);
    return lng ? launch_b8_gemm<128, true>(hd, ad, A, bd, B, D, ldd, args, stream)
               : launch_b8_gemm<128, false>(hd, ad, A, bd, B, D, ldd, args, stream);
}

// The workspace of sbl_b8_linear_backward: dY in both block orders and X
// transposed, each section 256-byte aligned.
struct BackwardPlan {
    sbl_b8_desc g, gt, xt;
    int64_t g_codes, g_scales, gt_codes, gt_scales, xt_codes, xt_scales, total;
};

static BackwardPlan backward_plan(int32_t O, int32_t K, int32_t T, int32_t g_type, int32_t x_type)
{
    BackwardPlan p;
    p.g = {T, O, g_type};
    p.gt = {O, T, g_type};
    p.xt = {K, T, x_type};
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += round_up(bytes, 256);
        return here;
    };
    p.g_codes = take(static_cast<int64_t>(T) * b8_ld(&p.g));
    p.g_scales = take(b8_scale_size(&p.g));
    p.gt_codes = take(static_cast<int64_t>(O) * b8_ld(&p.gt));
    p.gt_scales = take(b8_scale_size(&p.gt));
    p.xt_codes = take(static_cast<int64_t>(K) * b8_ld(&p.xt));
    p.xt_scales = take(b8_scale_size(&p.xt));
    p.total = at;
    return p;
}

// ------------------------------------------------------------------- norm --
template <int TYPE>
static sbl_status norm_checkpoint(const uint16_t *X, int32_t T, int32_t K, const uint16_t *g, double eps, int8_t *Xq, float *d,
                                  NormCkpt ck, cudaStream_t stream)
{
    // four chunks a thread up to 256 threads a row, eight beyond (16384 x 2048:
    // 44 us against 49; 16384 x 11008: 436 against 285)
    const int nc = K <= 256 * 4 * 8 ? 4 : 8;
    int rt = 32;
    while (rt * nc < K / 8) rt *= 2;
    switch (nc * 10000 + rt) {
#define SBL_CASE(R, C)                                                                                              \
    case C * 10000 + R: {                                                                                           \
        constexpr int rows = R >= 256 ? 1 : 256 / R;                                                                \
        return launch(act_norm_quant_kernel<R, TYPE, C>, ck.rp / rows, R > 256 ? R : 256, 0, stream, X, T, K, g,    \
                      eps, Xq, d, ck);                                                                              \
    }
        SBL_CASE(32, 4)
        SBL_CASE(64, 4)
        SBL_CASE(128, 4)
        SBL_CASE(256, 4)
        SBL_CASE(256, 8)
        SBL_CASE(512, 8)
        SBL_CASE(1024, 8)
#undef SBL_CASE
    }
    return SBL_ERR_SHAPE;
}

// Threads that share a row in the backward, one 16-element chunk each, and the
// CTAs a longer row is split over.
static int norm_row_threads(int32_t K)
{
    int rt = 32;
    while (rt < kNormLongThreads && rt < K / 16) rt *= 2;
    return rt;
}

static int norm_split(int32_t K)
{
    int split = 1;
    while (split * kNormLongThreads < K / 16) split *= 2;
    return split;
}

// Units (CTAs, or clusters for long rows) that go through the rows: the 512
// threads that fit an SM at 128 registers.
static int64_t norm_units(int32_t T, int32_t K, int num_sms)
{
    const int rt = norm_row_threads(K);
    const int rows = rt >= 256 ? 1 : 256 / rt, block = std::max(rt, 256);
    return std::min<int64_t>({(static_cast<int64_t>(T) + rows - 1) / rows, static_cast<int64_t>(512 / block) * num_sms / norm_split(K),
                              kNormPartials});
}

template <int TYPE>
static sbl_status norm_backward(NormBwdArgs a, int64_t units, cudaStream_t stream)
{
    a.split = norm_split(a.K);
    const int rt = norm_row_threads(a.K);
    const size_t smem = rt < 256 && a.partial ? static_cast<size_t>(a.K) * 4 : 0;
    switch (rt) {
    case 32: return launch(norm_backward_kernel<TYPE, 32>, units, 256, smem, stream, a);
    case 64: return launch(norm_backward_kernel<TYPE, 64>, units, 256, smem, stream, a);
    case 128: return launch(norm_backward_kernel<TYPE, 128>, units, 256, smem, stream, a);
    case 256: return launch(norm_backward_kernel<TYPE, 256>, units, 256, smem, stream, a);
    default: return launch_cluster(norm_backward_kernel<TYPE, kNormLongThreads>, units * a.split, a.split, kNormLongThreads, stream, a);
    }
}

// ------------------------------------------------------------- activation --
template <int TYPE, int ACT>
static sbl_status glu_forward(const HostDevice &hd, const GluFwdArgs &a, cudaStream_t stream)
{
    const int64_t rows = a.gc || a.uc ? a.rp : a.rows;  // padded rows have scales to write
    return a.U ? launch_walk(hd, glu_forward_kernel<TYPE, ACT, true>, rows, a, stream)
               : launch_walk(hd, glu_forward_kernel<TYPE, ACT, false>, rows, a, stream);
}

template <int TYPE, int ACT>
static sbl_status glu_backward(const HostDevice &hd, const GluBwdArgs &a, cudaStream_t stream)
{
    return a.uc ? launch_walk(hd, glu_backward_kernel<TYPE, ACT, true>, a.rows, a, stream)
                : launch_walk(hd, glu_backward_kernel<TYPE, ACT, false>, a.rows, a, stream);
}

}  // namespace sbl

using namespace sbl;

extern "C" {

size_t sbl_b8_row_bytes(const sbl_b8_desc *desc) { return check_b8(desc) == SBL_OK ? static_cast<size_t>(b8_ld(desc)) : 0; }

size_t sbl_b8_scale_bytes(const sbl_b8_desc *desc)
{
    return check_b8(desc) == SBL_OK ? static_cast<size_t>(b8_scale_size(desc)) : 0;
}

sbl_status sbl_b8_quantize(const sbl_b8_desc *desc, const void *X, int32_t x_is_fp32, int64_t ldx, sbl_b8_blocks blocks,
                           const sbl_b8 *out, const sbl_b8 *out_t, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if ((blocks != SBL_B8_ROWS && blocks != SBL_B8_TILES) || (!out && !out_t)) return SBL_ERR_INVALID_ARG;
    if (desc->rows == 0) return SBL_OK;
    if (!X || (out && !complete(out)) || (out_t && !complete(out_t))) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(X, ldx, desc->cols, x_is_fp32 ? 4 : 2)) != SBL_OK) return st;
    if ((out && !b8_aligned(out)) || (out_t && !b8_aligned(out_t))) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    return quantize(hd, desc, X, x_is_fp32 != 0, ldx, blocks == SBL_B8_TILES, out, out_t, static_cast<cudaStream_t>(stream));
}

sbl_status sbl_b8_transpose(const sbl_b8_desc *desc, const sbl_b8 *in, int32_t type_t, const sbl_b8 *out_t, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if (type_t != SBL_B8_E4M3 && type_t != SBL_B8_E5M2 && type_t != SBL_B8_I8) return SBL_ERR_INVALID_ARG;
    if (desc->rows == 0) return SBL_OK;
    if (!complete(in) || !complete(out_t)) return SBL_ERR_INVALID_ARG;
    if (!b8_aligned(in) || !b8_aligned(out_t)) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    return transpose(desc, in, type_t, out_t, false, static_cast<cudaStream_t>(stream));
}

sbl_status sbl_b8_dequantize(const sbl_b8_desc *desc, const sbl_b8 *in, uint16_t *X, int64_t ldx, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if (desc->rows == 0) return SBL_OK;
    if (!complete(in) || !X) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(X, ldx, desc->cols, 2)) != SBL_OK) return st;
    if (!b8_aligned(in)) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    B8ReadArgs a;
    memset(&a, 0, sizeof(a));
    a.codes = in->codes;
    a.ldc = b8_ld(desc);
    a.scales = scale_words(in);
    a.rp = b8_rp(desc->rows);
    a.rows = desc->rows;
    a.cols = desc->cols;
    a.words = b8_words(desc->cols);
    a.X = X;
    a.ldx = ldx;
    a.v32 = rows32(X, ldx);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (desc->type) {
    case SBL_B8_E4M3: return launch_walk(hd, b8_dequantize_kernel<kB8E4M3>, a.rows, a, s);
    case SBL_B8_E5M2: return launch_walk(hd, b8_dequantize_kernel<kB8E5M2>, a.rows, a, s);
    default: return launch_walk(hd, b8_dequantize_kernel<kB8I8>, a.rows, a, s);
    }
}

sbl_status sbl_b8_gemm(const sbl_b8_desc *a_desc, const sbl_b8 *a, const sbl_b8_desc *b_desc, const sbl_b8 *b, void *D, int64_t ldd,
                       int32_t d_is_fp32, int32_t accumulate, void *stream)
{
    sbl_status st = check_b8(a_desc);
    if (st != SBL_OK) return st;
    if ((st = check_b8(b_desc)) != SBL_OK) return st;
    if (a_desc->type == SBL_B8_I8 || b_desc->type == SBL_B8_I8) return SBL_ERR_UNSUPPORTED;
    if (a_desc->cols != b_desc->cols || b_desc->rows < 16 || b_desc->rows % 16 != 0) return SBL_ERR_SHAPE;
    if (accumulate && !d_is_fp32) return SBL_ERR_INVALID_ARG;
    if (a_desc->rows == 0) return SBL_OK;
    if (!complete(a) || !complete(b) || !D) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(D, ldd, b_desc->rows, d_is_fp32 ? 4 : 2)) != SBL_OK) return st;
    if (!b8_aligned(a) || !b8_aligned(b)) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    return gemm(hd, a_desc, a, b_desc, b, D, ldd, d_is_fp32 != 0, accumulate != 0, false, static_cast<cudaStream_t>(stream));
}

// W [O, K] of a b8 linear: both sizes multiples of 16 up to 65536, a product type.
static sbl_status check_b8_weight(const sbl_b8_desc *w)
{
    const sbl_status st = check_b8_act(w);
    if (st != SBL_OK) return st;
    if (w->type == SBL_B8_I8) return SBL_ERR_UNSUPPORTED;
    if (w->rows < 16 || w->rows % 16 != 0 || w->rows > kMaxDim) return SBL_ERR_SHAPE;
    return SBL_OK;
}

sbl_status sbl_b8_linear_forward(const sbl_b8_desc *w_desc, const sbl_b8 *w, const uint16_t *X, int64_t ldx, int32_t T, int32_t x_type,
                                 const sbl_b8 *xq, void *Y, int64_t ldy, int32_t y_is_fp32, void *stream)
{
    sbl_status st = check_b8_weight(w_desc);
    if (st != SBL_OK) return st;
    const sbl_b8_desc xd = {T, w_desc->cols, x_type};
    if ((st = check_b8(&xd)) != SBL_OK) return st;
    if (x_type == SBL_B8_I8) return SBL_ERR_UNSUPPORTED;
    if (T == 0) return SBL_OK;
    if (!complete(w) || !complete(xq) || !X || !Y) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(X, ldx, w_desc->cols, 2)) != SBL_OK) return st;
    if ((st = check_strided(Y, ldy, w_desc->rows, y_is_fp32 ? 4 : 2)) != SBL_OK) return st;
    if (!b8_aligned(w) || !b8_aligned(xq)) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One launch that quantises X itself while each CTA's share of it is
    // small, up to 112 (token, block) pairs; 120 measured even with two launches
    // (n x k: 6912 x 2560: 1 token, 5 pairs, 7.3 us against 9.1, 16 tokens, 80 pairs, 8.5
    // against 9.8, 24 tokens, 120 pairs, 10.4 against 10.2; 2560 x 6912: 16 tokens,
    // 112 pairs, 9.6 against 10.6).
    if (T <= 64) {
        const SkinnyPlan p = skinny_plan(hd.num_sms, w_desc->rows, w_desc->cols, T, true);
        if (p.smem <= kB8SmemAll && p.tmem_cols <= kTmemCols && static_cast<int64_t>(T) * p.max_blocks <= 112 && !(y_is_fp32 && p.max_blocks > kB8SegBlocks))
            return skinny(hd, p, w_desc, w, &xd, X, ldx, xq, Y, ldy, y_is_fp32 != 0, false, s);
    }
    if ((st = quantize(hd, &xd, X, false, ldx, false, xq, nullptr, s)) != SBL_OK) return st;
    return gemm(hd, &xd, xq, w_desc, w, Y, ldy, y_is_fp32 != 0, false, false, s);
}

size_t sbl_b8_linear_workspace_bytes(const sbl_b8_desc *w_desc, int32_t T)
{
    if (check_b8_weight(w_desc) != SBL_OK || T < 0 || T > kB8MaxRows) return 0;
    return static_cast<size_t>(backward_plan(w_desc->rows, w_desc->cols, T, SBL_B8_E4M3, SBL_B8_E4M3).total);
}

sbl_status sbl_b8_linear_backward(const sbl_b8_desc *w_desc, const sbl_b8 *w_t, const sbl_b8 *xq, int32_t x_type, const uint16_t *dY,
                                  int64_t lddy, int32_t T, int32_t g_type, void *dX, int32_t dx_is_fp32, float *dW,
                                  int32_t dw_accumulate, void *workspace, size_t workspace_bytes, void *stream)
{
    sbl_status st = check_b8_weight(w_desc);
    if (st != SBL_OK) return st;
    const int32_t O = w_desc->rows, K = w_desc->cols;
    const sbl_b8_desc xd = {T, K, x_type}, gd = {T, O, g_type};
    if ((st = check_b8(&xd)) != SBL_OK || (st = check_b8(&gd)) != SBL_OK) return st;
    if (x_type == SBL_B8_I8 || g_type == SBL_B8_I8) return SBL_ERR_UNSUPPORTED;
    if (!dX && !dW) return SBL_ERR_INVALID_ARG;
    if (dW && !aligned16(dW)) return SBL_ERR_ALIGNMENT;
    if (T > 0) {
        if (!dY || (dX && !complete(w_t)) || (dW && !complete(xq))) return SBL_ERR_INVALID_ARG;
        if ((st = check_strided(dY, lddy, O, 2)) != SBL_OK) return st;
        if ((dX && (!aligned16(dX) || !b8_aligned(w_t))) || (dW && !b8_aligned(xq))) return SBL_ERR_ALIGNMENT;
        if (!workspace || workspace_bytes < sbl_b8_linear_workspace_bytes(w_desc, T)) return SBL_ERR_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SBL_ERR_ALIGNMENT;
    }
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        return dW && !dw_accumulate ? launched(cudaMemsetAsync(dW, 0, static_cast<size_t>(O) * K * 4, s)) : SBL_OK;
    }
    const BackwardPlan p = backward_plan(O, K, T, g_type, x_type);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const sbl_b8 g = {ws + p.g_codes, ws + p.g_scales}, gt = {ws + p.gt_codes, ws + p.gt_scales}, xt = {ws + p.xt_codes, ws + p.xt_scales};
    if ((st = quantize(hd, &gd, dY, false, lddy, false, dX ? &g : nullptr, dW ? &gt : nullptr, s)) != SBL_OK) return st;
    // X's transpose needs nothing from the quantiser of dY before it, nor dW's
    // product from dX's: they start beside them (`late`), dW's tiles on the
    // SMs that dX's leave (the step of 777 x 1536 x 1536: 43 -> 35 us).
    if (dW && (st = transpose(&xd, xq, x_type, &xt, true, s)) != SBL_OK) return st;
    if (dX) {
        const sbl_b8_desc wt = {K, O, w_desc->type};
        if ((st = gemm(hd, &p.g, &g, &wt, w_t, dX, K, dx_is_fp32 != 0, false, false, s)) != SBL_OK) return st;
    }
    if (dW) return gemm(hd, &p.gt, &gt, &p.xt, &xt, dW, K, true, dw_accumulate != 0, dX != nullptr, s);
    return SBL_OK;
}

sbl_status sbl_glu_forward(const sbl_b8_desc *desc, sbl_activation act, const uint16_t *G, int64_t ldg, const uint16_t *U, int64_t ldu,
                           uint16_t *H, int64_t ldh, const sbl_b8 *g8, const sbl_b8 *u8, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if ((act != SBL_ACT_SILU && act != SBL_ACT_RELU2) || (!H && !g8 && !u8) || (u8 && !U)) return SBL_ERR_INVALID_ARG;
    if (desc->rows == 0) return SBL_OK;
    if (!G || (g8 && !complete(g8)) || (u8 && !complete(u8))) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(G, ldg, desc->cols, 2)) != SBL_OK || (U && (st = check_strided(U, ldu, desc->cols, 2)) != SBL_OK) ||
        (H && (st = check_strided(H, ldh, desc->cols, 2)) != SBL_OK))
        return st;
    if ((g8 && !b8_aligned(g8)) || (u8 && !b8_aligned(u8))) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    GluFwdArgs a;
    memset(&a, 0, sizeof(a));
    a.G = G;
    a.U = U;
    a.ldg = ldg;
    a.ldu = ldu;
    a.H = H;
    a.ldh = ldh;
    if (g8) a.gc = g8->codes, a.gs = scale_words(g8);
    if (u8) a.uc = u8->codes, a.us = scale_words(u8);
    a.ldc = b8_ld(desc);
    a.rp = b8_rp(desc->rows);
    a.rows = desc->rows;
    a.cols = desc->cols;
    a.words = b8_words(desc->cols);
    a.v32 = rows32(G, ldg) && rows32(U, ldu) && rows32(H, ldh);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (desc->type * 2 + act) {
    case SBL_B8_E4M3 * 2 + SBL_ACT_SILU: return glu_forward<kB8E4M3, kActSilu>(hd, a, s);
    case SBL_B8_E4M3 * 2 + SBL_ACT_RELU2: return glu_forward<kB8E4M3, kActRelu2>(hd, a, s);
    case SBL_B8_E5M2 * 2 + SBL_ACT_SILU: return glu_forward<kB8E5M2, kActSilu>(hd, a, s);
    case SBL_B8_E5M2 * 2 + SBL_ACT_RELU2: return glu_forward<kB8E5M2, kActRelu2>(hd, a, s);
    case SBL_B8_I8 * 2 + SBL_ACT_SILU: return glu_forward<kB8I8, kActSilu>(hd, a, s);
    default: return glu_forward<kB8I8, kActRelu2>(hd, a, s);
    }
}

sbl_status sbl_glu_backward(const sbl_b8_desc *desc, sbl_activation act, const sbl_b8 *g8, const sbl_b8 *u8, const uint16_t *dH,
                            int64_t lddh, uint16_t *dG, int64_t lddg, uint16_t *dU, int64_t lddu, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if ((act != SBL_ACT_SILU && act != SBL_ACT_RELU2) || (u8 != nullptr) != (dU != nullptr)) return SBL_ERR_INVALID_ARG;
    if (desc->rows == 0) return SBL_OK;
    if (!complete(g8) || (u8 && !complete(u8)) || !dH || !dG) return SBL_ERR_INVALID_ARG;
    if ((st = check_strided(dH, lddh, desc->cols, 2)) != SBL_OK || (st = check_strided(dG, lddg, desc->cols, 2)) != SBL_OK ||
        (dU && (st = check_strided(dU, lddu, desc->cols, 2)) != SBL_OK))
        return st;
    if (!b8_aligned(g8) || (u8 && !b8_aligned(u8))) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    GluBwdArgs a;
    memset(&a, 0, sizeof(a));
    a.gc = g8->codes;
    a.gs = scale_words(g8);
    if (u8) a.uc = u8->codes, a.us = scale_words(u8);
    a.ldc = b8_ld(desc);
    a.rp = b8_rp(desc->rows);
    a.dH = dH;
    a.ldh = lddh;
    a.dG = dG;
    a.ldg = lddg;
    a.dU = dU;
    a.ldu = lddu;
    a.rows = desc->rows;
    a.cols = desc->cols;
    a.words = b8_words(desc->cols);
    a.v32 = rows32(dH, lddh) && rows32(dG, lddg) && rows32(dU, lddu);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (desc->type * 2 + act) {
    case SBL_B8_E4M3 * 2 + SBL_ACT_SILU: return glu_backward<kB8E4M3, kActSilu>(hd, a, s);
    case SBL_B8_E4M3 * 2 + SBL_ACT_RELU2: return glu_backward<kB8E4M3, kActRelu2>(hd, a, s);
    case SBL_B8_E5M2 * 2 + SBL_ACT_SILU: return glu_backward<kB8E5M2, kActSilu>(hd, a, s);
    case SBL_B8_E5M2 * 2 + SBL_ACT_RELU2: return glu_backward<kB8E5M2, kActRelu2>(hd, a, s);
    case SBL_B8_I8 * 2 + SBL_ACT_SILU: return glu_backward<kB8I8, kActSilu>(hd, a, s);
    default: return glu_backward<kB8I8, kActRelu2>(hd, a, s);
    }
}

sbl_status sbl_quantize_act_rmsnorm_checkpoint(const sbl_b8_desc *desc, const uint16_t *X, const uint16_t *g, double eps, int8_t *Xq,
                                               float *d, const sbl_b8 *x8, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    if (desc->rows == 0) return SBL_OK;
    if (!X || !Xq || !d || !complete(x8)) return SBL_ERR_INVALID_ARG;
    if (!(eps >= 0.0) || eps > 3.0e38) return SBL_ERR_INVALID_ARG;  // finite, non-negative
    if (!aligned16(X) || !aligned16(Xq) || !aligned16(d) || (g && !aligned16(g)) || !b8_aligned(x8)) return SBL_ERR_ALIGNMENT;
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    NormCkpt ck;
    ck.codes = x8->codes;
    ck.scales = scale_words(x8);
    ck.rp = b8_rp(desc->rows);
    ck.words = b8_words(desc->cols);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (desc->type) {
    case SBL_B8_E4M3: return norm_checkpoint<kB8E4M3>(X, desc->rows, desc->cols, g, eps, Xq, d, ck, s);
    case SBL_B8_E5M2: return norm_checkpoint<kB8E5M2>(X, desc->rows, desc->cols, g, eps, Xq, d, ck, s);
    default: return norm_checkpoint<kB8I8>(X, desc->rows, desc->cols, g, eps, Xq, d, ck, s);
    }
}

size_t sbl_rmsnorm_backward_workspace_bytes(int32_t T, int32_t K)
{
    if (T < 0 || K < 16 || K % 16 != 0 || K > kMaxDim) return 0;
    return static_cast<size_t>(round_up(std::min<int64_t>(std::max(T, 1), kNormPartials) * K * 4, 256));
}

sbl_status sbl_rmsnorm_backward(const sbl_b8_desc *desc, const sbl_b8 *x8, const uint16_t *g, double eps, const uint16_t *dU,
                                const uint16_t *dR, uint16_t *dX, float *dg, void *workspace, size_t workspace_bytes, void *stream)
{
    sbl_status st = check_b8_act(desc);
    if (st != SBL_OK) return st;
    const int32_t T = desc->rows, K = desc->cols;
    if (!(eps >= 0.0) || eps > 3.0e38 || (dg && !g)) return SBL_ERR_INVALID_ARG;
    if ((g && !aligned16(g)) || (dg && !aligned16(dg))) return SBL_ERR_ALIGNMENT;
    if (T > 0) {
        if (!complete(x8) || !dU || !dX) return SBL_ERR_INVALID_ARG;
        if (!b8_aligned(x8) || !aligned16(dU) || !aligned16(dX) || (dR && !aligned16(dR))) return SBL_ERR_ALIGNMENT;
        if (dg && (!workspace || workspace_bytes < sbl_rmsnorm_backward_workspace_bytes(T, K))) return SBL_ERR_WORKSPACE;
        if (dg && (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SBL_ERR_ALIGNMENT;
    }
    HostDevice hd;
    if ((st = b8_device(&hd)) != SBL_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        return dg ? launched(cudaMemsetAsync(dg, 0, static_cast<size_t>(K) * 4, s)) : SBL_OK;
    }
    NormBwdArgs a;
    memset(&a, 0, sizeof(a));
    a.xc = x8->codes;
    a.xs = scale_words(x8);
    a.ldc = K;
    a.rp = b8_rp(T);
    a.gain = g;
    a.dU = dU;
    a.dR = dR;
    a.dX = dX;
    a.partial = dg ? static_cast<float *>(workspace) : nullptr;
    a.T = T;
    a.K = K;
    a.v32 = rows32(dU, K) && rows32(dR, K) && rows32(dX, K);
    // eps = q 2^(2 (e - 127)), 1/4 <= q < 1
    int exp2 = -2 * 1024;
    const double frac = eps > 0.0 ? frexp(eps, &exp2) : 0.0;
    const int half = (exp2 + 2049) / 2 - 1024;  // ceil(exp2 / 2)
    a.eps_q = static_cast<float>(ldexp(frac, exp2 - 2 * half));
    a.eps_e = half + 127;
    const int64_t units = norm_units(T, K, hd.num_sms);
    switch (desc->type) {
    case SBL_B8_E4M3: st = norm_backward<kB8E4M3>(a, units, s); break;
    case SBL_B8_E5M2: st = norm_backward<kB8E5M2>(a, units, s); break;
    default: st = norm_backward<kB8I8>(a, units, s); break;
    }
    if (st != SBL_OK || !dg) return st;
    return launch(norm_dgain_kernel, (K + 31) / 32, 1024, 0, s, static_cast<const float *>(a.partial), static_cast<int32_t>(units), K, dg);
}

}  // extern "C"
