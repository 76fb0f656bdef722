// w4.cu — entry points of the products with 4-bit weights: argument validation and
// launches of the kernels of w4.cuh.  See include/qmoe.h for the contract of every
// function.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "../../include/qmoe.h"
#include "host.cuh"
#include "w4.cuh"
#include "w4_many.cuh"
#include "w4_rule.cuh"

namespace qmoe {

constexpr int64_t W4_MAX_COLS = 1 << 20;
constexpr int64_t W4_MAX_ROWS = 0x7fffff00;
constexpr int W4_MAX_GROUPS = 1024;
constexpr int64_t W4_MAX_TILES = 0x7fff0000;  // an int counts them, one grid past the last

static int w4_size(int t) { return t == QMOE_F32 ? 4 : t == QMOE_BF16 || t == QMOE_F16 ? 2 : 0; }

static qmoe_status too_many_tiles(const w4::Params& p) {
    return fail(QMOE_ERR_UNSUPPORTED, "4-bit product: %d rows of W times %d of x in %d groups are too "
                "many", p.N, p.M, p.E);
}

// The kernel for few rows: tiles of 16 weight rows and as many tokens as NB MMA column
// blocks of eight hold.
template <class X, int S, int NB>
static qmoe_status launch_few(w4::Params p, const DevInfo& d, cudaStream_t st) {
    constexpr int parts = std::is_same<X, float>::value ? 3 : 1;
    p.nt = 8 * NB / parts;
    p.cols = std::min(p.nt, p.M) * parts;
    const int units = (p.K + w4::UNIT - 1) / w4::UNIT;
    const int unit_bytes = p.cols * w4::UNIT * 2;
    const int room = d.smem_pair - 512;
    // K over the CTAs of a cluster: until x fits, and further while the tiles leave SMs
    // idle; a CTA's part over its warps, a block of four units each
    int ranks = 1, smem = 0;
    for (int r = 1; r <= w4::MAX_RANKS && r <= units; r *= 2) {
        w4::Params q = p;
        q.rank_units = (units + r - 1) / r;
        const int blocks = (q.rank_units + w4::BLOCK - 1) / w4::BLOCK;
        q.wk = 1;
        // (no more parts than a round's x leaves room for)
        while (q.wk < w4::WARPS && q.wk < blocks && 2 * q.wk * w4::BLOCK * unit_bytes <= room / 5 * 3)
            q.wk *= 2;
        const int rows = 16 * w4::WARPS / q.wk;
        q.nb = (q.N + rows - 1) / rows;
        q.slot = r > 1 ? rows * q.nt : 0;
        const int fixed = w4::few_fixed(q.E, NB, q.slot * r);
        const int round_bytes = q.wk * w4::BLOCK * unit_bytes;
        const int rounds = (blocks + q.wk - 1) / q.wk;
        if (fixed + round_bytes > room) break;
        q.pass_rounds = std::min(rounds, (room - fixed) / round_bytes);
        p = q;
        ranks = r;
        smem = fixed + q.pass_rounds * round_bytes;
        const bool full = gmm::max_tiles(q.M, q.E, q.nt, q.nb) * 2 * r > 2 * d.sms;
        if (q.pass_rounds == rounds && (full || blocks <= w4::WARPS)) break;
    }
    const int64_t tiles = gmm::max_tiles(p.M, p.E, p.nt, p.nb);
    if (tiles > W4_MAX_TILES) return too_many_tiles(p);
    p.tiles = static_cast<int>(tiles);
    for (p.rts_log = 0; (p.wk << p.rts_log) < w4::WARPS;) ++p.rts_log;
    auto kern = w4::few_kernel<X, S, NB>;
    static std::atomic<bool> configured[64];
    if (!configured[d.dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(4-bit product)");
        configured[d.dev].store(true);
    }
    const int clusters = static_cast<int>(std::min<int64_t>(tiles, 2 * d.sms / ranks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
    cfg.blockDim = dim3(w4::THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return cuda_fail(e, "4-bit product launch");
    return QMOE_OK;
}

static qmoe_status tensor_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base,
                              const cuuint64_t* dims, const cuuint64_t* strides,
                              const cuuint32_t* box) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(QMOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t estride[3] = {1, 1, 1};
    const CUresult r = fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estride,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(QMOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return QMOE_OK;
}
// The codes as [E][N][K / 2] bytes, boxes of 256 rows by 128 bytes.
static qmoe_status codes_map(CUtensorMap* m, const w4::Params& p) {
    const cuuint64_t row = static_cast<cuuint64_t>(p.K / 2);
    const cuuint64_t dims[3] = {row, static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.E)};
    const cuuint64_t strides[2] = {row, row * static_cast<cuuint64_t>(p.N)};
    const cuuint32_t box[3] = {128, w4::MANY_ROWS, 1};
    return tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.W, dims, strides, box);
}
// 16-bit token rows, boxes of 64 rows by 64 columns.
static qmoe_status rows_map(CUtensorMap* m, const w4::Params& p, bool bf16) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.K), static_cast<cuuint64_t>(p.M)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.ldx) * 2};
    const cuuint32_t box[2] = {64, w4::MANY_NT};
    return tensor_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      2, p.x, dims, strides, box);
}

// The kernel for many rows: a CTA per SM, or clusters that share K while the tiles are
// fewer.
template <class C>
static qmoe_status launch_many(w4::Params p, const DevInfo& d, cudaStream_t st) {
    static_assert(C::smem(W4_MAX_GROUPS) + 256 <= 232448, "shared memory, static arrays included");
    auto kern = w4::many_kernel<C>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(C::smem(p.E));
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // clusters of two, four and eight that the GPU holds at once
    static std::atomic<int> fit[64][3];
    static std::atomic<bool> configured[64];
    if (!configured[d.dev].load()) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::smem(W4_MAX_GROUPS));
        cfg.numAttrs = 1;
        for (int i = 0; i < 3 && e == cudaSuccess; ++i) {
            int n = 0;
            attr[0].val.clusterDim.x = 2u << i;
            cfg.gridDim = dim3(2u << i);
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            fit[d.dev][i].store(n);
        }
        if (e != cudaSuccess) return cuda_fail(e, "setting up the 4-bit product");
        configured[d.dev].store(true);
    }
    CUtensorMap tw, tx;
    if (qmoe_status s = codes_map(&tw, p)) return s;
    tx = tw;
    if constexpr (C::TMA_X)
        if (qmoe_status s = rows_map(&tx, p, std::is_same<typename C::X, __nv_bfloat16>::value))
            return s;
    p.nb = (p.N + w4::MANY_ROWS - 1) / w4::MANY_ROWS;
    const int64_t tiles = gmm::max_tiles(p.M, p.E, w4::MANY_NT, p.nb);
    if (tiles > W4_MAX_TILES) return too_many_tiles(p);
    const int kb = (p.K + 127) / 128;
    int ranks = 1;
    for (int i = 0; i < 3 && tiles <= fit[d.dev][i].load() && (2 << i) <= kb; ++i) ranks = 2 << i;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(static_cast<unsigned>(
        ranks > 1 ? tiles * ranks : std::min<int64_t>(tiles, d.sms)));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, tw, tx);
    if (e != cudaSuccess) return cuda_fail(e, "4-bit product launch");
    return QMOE_OK;
}

template <class X, int S>
static qmoe_status launch_rows(const w4::Params& p, const DevInfo& d, cudaStream_t st) {
    constexpr int one = std::is_same<X, float>::value ? 2 : 8;  // tokens of one column block
    const int64_t groups = std::min(p.M, p.E);
    if (w4::many_rows(p.M, p.E, p.N, p.K, std::is_same<X, float>::value)) {
        if constexpr (!std::is_same<X, float>::value)
            if (p.vec_x) return launch_many<w4::Many<X, S, true>>(p, d, st);
        return launch_many<w4::Many<X, S, false>>(p, d, st);
    }
    return p.M <= one * groups ? launch_few<X, S, 1>(p, d, st) : launch_few<X, S, 2>(p, d, st);
}

template <class X>
static qmoe_status launch_scales(const w4::Params& p, const DevInfo& d, cudaStream_t st) {
    return p.S == 32   ? launch_rows<X, 32>(p, d, st)
           : p.S == 64 ? launch_rows<X, 64>(p, d, st)
                       : launch_rows<X, 128>(p, d, st);
}

static qmoe_status w4_run(const char* fn, const void* W, int stype, const void* scale,
                          const uint8_t* zero, int32_t scale_cols, int32_t num_groups,
                          int64_t rows, int64_t cols, int xtype, const void* x, int64_t n_rows,
                          int64_t ldx, const int32_t* offsets, int ytype, void* y, int64_t ldy,
                          void* stream) {
    if (!w4_size(stype) || !w4_size(xtype) || !w4_size(ytype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: scale, x and y types %d, %d, %d must be F32, BF16 or "
                    "F16", fn, stype, xtype, ytype);
    if (rows <= 0 || cols <= 0 || n_rows < 0 || ldx < cols || ldy < rows)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: rows=%lld, cols=%lld >= 1, n=%lld >= 0, ldx=%lld >= cols and ldy=%lld >= "
                    "rows are needed",
                    fn, (long long)rows, (long long)cols, (long long)n_rows, (long long)ldx,
                    (long long)ldy);
    if (scale_cols != 32 && scale_cols != 64 && scale_cols != 128)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: scale_cols=%d is not 32, 64 or 128", fn, scale_cols);
    if (cols % scale_cols)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: cols=%lld is not a multiple of scale_cols=%d",
                    fn, (long long)cols, scale_cols);
    if (rows > W4_MAX_ROWS || n_rows > W4_MAX_ROWS || cols > W4_MAX_COLS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: rows=%lld, n=%lld or cols=%lld is too large", fn,
                    (long long)rows, (long long)n_rows, (long long)cols);
    if (n_rows == 0) return QMOE_OK;
    if (!W || !scale || !x || !y)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer (W, scale, x or y)", fn);
    if (!aligned(W, 16) || !aligned(scale, w4_size(stype)) || !aligned(x, w4_size(xtype)) ||
        !aligned(y, w4_size(ytype)))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: W must be 16-byte aligned, scale, x and y aligned to their elements", fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    w4::Params p = {};
    p.W = static_cast<const uint8_t*>(W);
    p.scale = scale;
    p.zero = zero;
    p.x = x;
    p.y = y;
    p.offsets = offsets;
    p.ldx = ldx;
    p.ldy = ldy;
    p.M = static_cast<int>(n_rows);
    p.N = static_cast<int>(rows);
    p.K = static_cast<int>(cols);
    p.E = num_groups;
    p.S = scale_cols;
    p.stype = stype;
    p.ytype = ytype;
    p.vec_x = aligned(x, 16) && (ldx * w4_size(xtype)) % 16 == 0;
    p.err = d->err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return xtype == QMOE_F32    ? launch_scales<float>(p, *d, st)
           : xtype == QMOE_BF16 ? launch_scales<__nv_bfloat16>(p, *d, st)
                                : launch_scales<__half>(p, *d, st);
}

}  // namespace qmoe

using namespace qmoe;

// ====================================================================== C ABI
extern "C" {

qmoe_status w4_mm(const void* W, int stype, const void* scale, const uint8_t* zero,
                  int32_t scale_cols, int64_t rows, int64_t cols, int xtype, const void* x,
                  int64_t n_tokens, int64_t ldx, int ytype, void* y, int64_t ldy, void* stream) {
    clear_error();
    return w4_run("w4_mm", W, stype, scale, zero, scale_cols, 1, rows, cols, xtype, x, n_tokens,
                  ldx, nullptr, ytype, y, ldy, stream);
}

qmoe_status w4_mm_grouped(const void* W, int stype, const void* scale, const uint8_t* zero,
                          int32_t scale_cols, int32_t num_groups, int64_t rows, int64_t cols,
                          int xtype, const void* x, int64_t n_rows, int64_t ldx,
                          const int32_t* offsets, int ytype, void* y, int64_t ldy, void* stream) {
    clear_error();
    const char* fn = "w4_mm_grouped";
    if (num_groups <= 0)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: num_groups=%d must be >= 1", fn, num_groups);
    if (num_groups > W4_MAX_GROUPS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: num_groups=%d exceeds %d", fn, num_groups,
                    W4_MAX_GROUPS);
    if (n_rows > 0 && (!offsets || !aligned(offsets, 4)))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: offsets null or not 4-byte aligned", fn);
    return w4_run(fn, W, stype, scale, zero, scale_cols, num_groups, rows, cols, xtype, x, n_rows,
                  ldx, offsets, ytype, y, ldy, stream);
}

}  // extern "C"
