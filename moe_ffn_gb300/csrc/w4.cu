// w4.cu — entry points of the products with 4-bit weights: argument validation and
// launches of the kernels of w4.cuh.  See include/qmoe.h for the contract of every
// function.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/qmoe.h"
#include "host.cuh"
#include "w4.cuh"

namespace qmoe {

constexpr int64_t W4_MAX_COLS = 1 << 20;
constexpr int64_t W4_MAX_ROWS = 0x7fffff00;
constexpr int W4_MAX_GROUPS = 1024;

static int w4_size(int t) { return t == QMOE_F32 ? 4 : t == QMOE_BF16 || t == QMOE_F16 ? 2 : 0; }

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
    p.xtype = xtype;
    p.ytype = ytype;
    p.err = d->err;
    const int64_t items = (n_rows * rows + w4::THREADS / 32 - 1) / (w4::THREADS / 32);
    const cudaError_t e = launch_pdl(
        w4::mm_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, d->sms * 8))),
        dim3(w4::THREADS), 0, static_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return cuda_fail(e, "4-bit product launch");
    return QMOE_OK;
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
