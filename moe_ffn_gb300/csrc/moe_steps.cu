// moe_steps.cu — entry points of the steps around a mixture-of-experts layer's
// products: argument validation and launches of the kernels of moe_steps.cuh.  See
// include/qmoe.h for the contract of every function.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/qmoe.h"
#include "host.cuh"
#include "moe_steps.cuh"

namespace qmoe {

constexpr int64_t MAX_STEP_COLS = 1 << 20;
constexpr int64_t MAX_PAIRS = 1 << 25;  // n_tokens * top_k

static int float_size(int t) { return t == QMOE_F32 ? 4 : t == QMOE_BF16 || t == QMOE_F16 ? 2 : 0; }

// Calls f with a value of the type that `type` names.
template <class F>
static auto with_type(int type, F&& f) {
    return type == QMOE_F32 ? f(float()) : type == QMOE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

// ------------------------------------------------------------------- routing
static qmoe_status route_check(const char* fn, int ltype, const void* logits, int64_t n_tokens,
                               int32_t num_experts, int64_t ldl, int32_t top_k,
                               int32_t route_flags) {
    if (!float_size(ltype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: logits type %d is not F32, BF16 or F16", fn, ltype);
    if (n_tokens < 0 || num_experts <= 0 || top_k <= 0 || top_k > num_experts || ldl < num_experts)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: n_tokens=%lld >= 0, num_experts=%d >= 1, 1 <= top_k=%d <= num_experts and "
                    "ldl=%lld >= num_experts are needed",
                    fn, (long long)n_tokens, num_experts, top_k, (long long)ldl);
    if (route_flags & ~QMOE_ROUTE_NO_RENORM)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: unknown route_flags=0x%x", fn,
                    static_cast<unsigned>(route_flags));
    if (num_experts > steps::MAX_EXPERTS || top_k > steps::MAX_TOPK)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: num_experts=%d > %d or top_k=%d > %d", fn,
                    num_experts, steps::MAX_EXPERTS, top_k, steps::MAX_TOPK);
    if (n_tokens > MAX_PAIRS / top_k)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: n_tokens * top_k exceeds %lld", fn,
                    (long long)MAX_PAIRS);
    if (n_tokens && (!logits || !aligned(logits, float_size(ltype))))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: logits null or not aligned to their elements", fn);
    return QMOE_OK;
}

// Whether a lane's run of V values of every row is whole and aligned to its size
// (16 bytes at most), so that it is loaded or stored as such.
static bool whole_runs(const void* p, int64_t ld, int size, int E, int V) {
    const int unit = std::min(16, V * size);
    return E % V == 0 && aligned(p, unit) && (ld * size) % unit == 0;
}

template <class T, int V>
static cudaError_t launch_route(steps::RouteParams p, cudaStream_t st) {
    p.vec = whole_runs(p.logits, p.ldl, sizeof(T), p.E, V);
    p.vec_g = p.grad && whole_runs(p.grad, p.ldg, sizeof(T), p.E, V);
    const dim3 grid(static_cast<unsigned>((p.n_tokens + steps::R_WARPS - 1) / steps::R_WARPS));
    return p.grad ? launch_pdl(steps::route_backward_kernel<T, V>, grid, dim3(steps::R_WARPS * 32),
                               0, st, p)
                  : launch_pdl(steps::route_kernel<T, V>, grid, dim3(steps::R_WARPS * 32), 0, st, p);
}

static qmoe_status run_route(const steps::RouteParams& p, int ltype, cudaStream_t st) {
    const cudaError_t e = with_type(ltype, [&](auto v) {
        using T = decltype(v);
        return p.E <= 32    ? launch_route<T, 1>(p, st)
               : p.E <= 64  ? launch_route<T, 2>(p, st)
               : p.E <= 128 ? launch_route<T, 4>(p, st)
               : p.E <= 256 ? launch_route<T, 8>(p, st)
               : p.E <= 512 ? launch_route<T, 16>(p, st)
                            : launch_route<T, 32>(p, st);
    });
    if (e != cudaSuccess) return cuda_fail(e, "routing launch");
    return QMOE_OK;
}

// ------------------------------------------------------------------- permute
// Tokens of a run and number of runs: 16 tokens, more where there would be more
// than 304 runs (two CTAs on each of 152 SMs), but never more pairs than a 16-bit
// count holds.
static void permute_runs(int64_t n_tokens, int top_k, int* run, int* runs) {
    const int64_t want = std::max<int64_t>(16, (n_tokens + 303) / 304);
    *run = static_cast<int>(std::min<int64_t>(want, 65535 / top_k));
    *runs = static_cast<int>((n_tokens + *run - 1) / *run);
}

static qmoe_status permute_check(const char* fn, int64_t n_tokens, int32_t num_experts,
                                 int32_t top_k) {
    if (n_tokens < 0 || num_experts <= 0 || top_k <= 0)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: n_tokens=%lld >= 0, num_experts=%d >= 1 and top_k=%d >= 1 are needed", fn,
                    (long long)n_tokens, num_experts, top_k);
    if (num_experts > steps::MAX_EXPERTS || top_k > steps::MAX_TOPK)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: num_experts=%d > %d or top_k=%d > %d", fn,
                    num_experts, steps::MAX_EXPERTS, top_k, steps::MAX_TOPK);
    if (n_tokens > MAX_PAIRS / top_k)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: n_tokens * top_k exceeds %lld", fn,
                    (long long)MAX_PAIRS);
    return QMOE_OK;
}

static size_t permute_ws(int64_t n_tokens, int32_t num_experts, int32_t top_k) {
    if (n_tokens * top_k <= steps::P_ALONE) return 256;
    int run, runs;
    permute_runs(n_tokens, top_k, &run, &runs);
    return (static_cast<size_t>(runs) * ((num_experts + 7) / 8 * 8) * 2 + 255) / 256 * 256;
}

template <int VB, bool STREAM>
static cudaError_t launch_permute(steps::PermuteParams p, int64_t row_bytes, dim3 grid, size_t smem,
                                  cudaStream_t st) {
    p.nvec = static_cast<int>(row_bytes / VB);
    return launch_pdl(steps::permute_kernel<VB, STREAM>, grid, dim3(steps::P_THREADS), smem, st, p);
}

// ------------------------------------------------------------------- combine
static qmoe_status combine_check(const char* fn, int ytype, const void* y, int64_t n_rows,
                                 int64_t cols, int64_t ldy, const int32_t* pos, const float* w,
                                 int64_t n_tokens, int32_t top_k, int otype, int64_t ldo) {
    if (!float_size(ytype) || !float_size(otype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: types %d and %d must be F32, BF16 or F16", fn, ytype,
                    otype);
    if (n_tokens < 0 || n_rows < 0 || cols <= 0 || top_k <= 0 || ldy < cols || ldo < cols)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: n_tokens=%lld >= 0, n_rows=%lld >= 0, top_k=%d >= 1, cols=%lld >= 1 and "
                    "row distances %lld, %lld >= cols are needed",
                    fn, (long long)n_tokens, (long long)n_rows, top_k, (long long)cols,
                    (long long)ldy, (long long)ldo);
    if (top_k > steps::MAX_TOPK || cols > MAX_STEP_COLS || n_rows > 0x7fffffff)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: top_k=%d > %d, cols=%lld > %lld or n_rows=%lld", fn,
                    top_k, steps::MAX_TOPK, (long long)cols, (long long)MAX_STEP_COLS,
                    (long long)n_rows);
    if (n_tokens > MAX_PAIRS / top_k)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: n_tokens * top_k exceeds %lld", fn,
                    (long long)MAX_PAIRS);
    if (n_tokens == 0) return QMOE_OK;
    if (!pos || (n_rows && !y))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer (pos or the rows)", fn);
    if (!aligned(pos, 4) || !aligned(w, 4) || !aligned(y, float_size(ytype)))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: pos, weights and rows must be aligned to their elements", fn);
    return QMOE_OK;
}

// Whether every row of an array is made of whole aligned 16-byte units.
static bool whole_units(const void* p, int64_t ld, int size) {
    return aligned(p, 16) && (ld * size) % 16 == 0;
}

template <class Y, class O, int N>
static cudaError_t launch_combine(const steps::CombineParams& p, int64_t n_tokens,
                                  cudaStream_t st) {
    if (p.grad_out)
        return launch_pdl(steps::combine_backward_kernel<Y, O, N>,
                          dim3(static_cast<unsigned>(n_tokens)), dim3(steps::C_THREADS), 0, st, p);
    const int per = steps::SUM_GROUPS<N> * steps::SUM_THREADS<N> * N;
    return launch_pdl(steps::combine_kernel<Y, O, N>,
                      dim3(static_cast<unsigned>(n_tokens), (p.cols + per - 1) / per),
                      dim3(steps::SUM_THREADS<N>), 0, st, p);
}

static qmoe_status run_combine(const steps::CombineParams& p, int ytype, int otype,
                               int64_t n_tokens, cudaStream_t st) {
    const int ys = float_size(ytype), os = float_size(otype);
    const bool vec = p.cols % 8 == 0 && whole_units(p.y, p.ldy, ys) &&
                     whole_units(p.grad_y, p.ldg, ys) && whole_units(p.residual, p.ldo, os) &&
                     whole_units(p.out, p.ldo, os) && whole_units(p.grad_out, p.ldo, os);
    const cudaError_t e = with_type(ytype, [&](auto y) {
        return with_type(otype, [&](auto o) {
            using Y = decltype(y);
            using O = decltype(o);
            return vec ? launch_combine<Y, O, 8>(p, n_tokens, st)
                       : launch_combine<Y, O, 1>(p, n_tokens, st);
        });
    });
    if (e != cudaSuccess) return cuda_fail(e, "combine launch");
    return QMOE_OK;
}

}  // namespace qmoe

using namespace qmoe;

// ====================================================================== C ABI
extern "C" {

qmoe_status moe_route(int ltype, const void* logits, int64_t n_tokens, int32_t num_experts,
                      int64_t ldl, int32_t top_k, int32_t route_flags, int32_t* topk_idx,
                      float* topk_w, void* stream) {
    clear_error();
    const char* fn = "moe_route";
    if (qmoe_status s = route_check(fn, ltype, logits, n_tokens, num_experts, ldl, top_k,
                                    route_flags))
        return s;
    if (n_tokens == 0) return QMOE_OK;
    if (!topk_idx || !topk_w || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: topk_idx or topk_w null or not 4-byte aligned",
                    fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    steps::RouteParams p = {};
    p.logits = logits;
    p.ldl = ldl;
    p.n_tokens = n_tokens;
    p.E = num_experts;
    p.k = top_k;
    p.renorm = !(route_flags & QMOE_ROUTE_NO_RENORM);
    p.idx = topk_idx;
    p.w = topk_w;
    return run_route(p, ltype, static_cast<cudaStream_t>(stream));
}

qmoe_status moe_route_backward(int ltype, const void* logits, int64_t n_tokens,
                               int32_t num_experts, int64_t ldl, int32_t top_k,
                               int32_t route_flags, const int32_t* topk_idx, const float* topk_w,
                               const float* grad_w, void* grad_logits, int64_t ldg, void* stream) {
    clear_error();
    const char* fn = "moe_route_backward";
    if (qmoe_status s = route_check(fn, ltype, logits, n_tokens, num_experts, ldl, top_k,
                                    route_flags))
        return s;
    if (ldg < num_experts)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: ldg=%lld must be >= num_experts=%d", fn,
                    (long long)ldg, num_experts);
    if (n_tokens == 0) return QMOE_OK;
    if (!topk_idx || !topk_w || !grad_w || !grad_logits)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer", fn);
    if (!aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(grad_w, 4) ||
        !aligned(grad_logits, float_size(ltype)))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: arrays must be aligned to their elements", fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    steps::RouteParams p = {};
    p.logits = logits;
    p.ldl = ldl;
    p.n_tokens = n_tokens;
    p.E = num_experts;
    p.k = top_k;
    p.renorm = !(route_flags & QMOE_ROUTE_NO_RENORM);
    p.idx = const_cast<int32_t*>(topk_idx);  // (read only where grad is set)
    p.w = const_cast<float*>(topk_w);
    p.grad_w = grad_w;
    p.grad = grad_logits;
    p.ldg = ldg;
    return run_route(p, ltype, static_cast<cudaStream_t>(stream));
}

size_t moe_permute_workspace_size(int64_t n_tokens, int32_t num_experts, int32_t top_k) {
    clear_error();
    if (permute_check("moe_permute", n_tokens, num_experts, top_k)) return 0;
    return permute_ws(n_tokens, num_experts, top_k);
}

qmoe_status moe_permute(int xtype, const void* x, int64_t n_tokens, int64_t cols, int64_t ldx,
                        const int32_t* topk_idx, int32_t num_experts, int32_t top_k, void* rows,
                        int64_t ldr, int32_t* offsets, int32_t* pos, void* ws, size_t ws_bytes,
                        void* stream) {
    clear_error();
    const char* fn = "moe_permute";
    const int size = float_size(xtype);
    if (!size)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: x type %d is not F32, BF16 or F16", fn, xtype);
    if (qmoe_status s = permute_check(fn, n_tokens, num_experts, top_k)) return s;
    if (cols <= 0 || ldx < cols || ldr < cols)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: cols=%lld >= 1, ldx=%lld >= cols and ldr=%lld >= cols are needed", fn,
                    (long long)cols, (long long)ldx, (long long)ldr);
    if (cols > MAX_STEP_COLS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: cols=%lld > %lld", fn, (long long)cols,
                    (long long)MAX_STEP_COLS);
    if (!offsets || !aligned(offsets, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: offsets null or not 4-byte aligned", fn);
    if (n_tokens && (!x || !topk_idx || !rows || !pos || !ws))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer", fn);
    if (!aligned(x, size) || !aligned(rows, size) || !aligned(topk_idx, 4) || !aligned(pos, 4) ||
        !aligned(ws, 16))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: arrays must be aligned to their elements, ws to 16 bytes", fn);
    const size_t need = permute_ws(n_tokens, num_experts, top_k);
    if (n_tokens && ws_bytes < need)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    steps::PermuteParams p = {};
    p.x = static_cast<const uint8_t*>(x);
    p.ldx = ldx * size;
    p.rows = static_cast<uint8_t*>(rows);
    p.ldr = ldr * size;
    p.idx = topk_idx;
    p.offsets = offsets;
    p.pos = pos;
    p.P = static_cast<int>(n_tokens * top_k);
    p.E = num_experts;
    p.Ep = (num_experts + 7) / 8 * 8;
    p.k = top_k;
    if (p.P > steps::P_ALONE) {
        permute_runs(n_tokens, top_k, &p.run, &p.runs);
        p.counts = static_cast<uint16_t*>(ws);
        const cudaError_t e = launch_pdl(steps::count_kernel, dim3(p.runs), dim3(steps::P_THREADS),
                                         static_cast<size_t>(p.Ep) * 4, st, p);
        if (e != cudaSuccess) return cuda_fail(e, "count launch");
    } else {
        p.run = static_cast<int>(std::max<int64_t>(1, (n_tokens + 2 * d->sms - 1) / (2 * d->sms)));
        p.runs = static_cast<int>(std::max<int64_t>(1, (n_tokens + p.run - 1) / p.run));
    }
    const int64_t row_bytes = cols * size;
    auto units = [&](int b) {
        return aligned(x, b) && aligned(rows, b) && row_bytes % b == 0 && p.ldx % b == 0 &&
               p.ldr % b == 0;
    };
    // Rows of more than half of L2 are written as a stream, evicted first: 4096 x 2048 top-8
    // (134 MB) 29.8 -> 27.3 us, 16384 x 1024 (268 MB) 57.7 -> 53.0; fewer take as long either
    // way and may still be there for the product that reads them.
    const bool past_l2 = static_cast<int64_t>(p.P) * row_bytes > (int64_t{64} << 20);
    // few runs: several CTAs share a run's columns (and each finds its rows)
    const int64_t segs = (row_bytes / 16 + 127) / 128 * p.run;
    const int share = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>(d->sms / p.runs, (segs + steps::P_WARPS - 1) / steps::P_WARPS)));
    const dim3 grid(p.runs, share);
    const size_t smem = static_cast<size_t>(steps::P_WARPS + 2) * p.Ep * 4;
    const cudaError_t e =
        units(16) ? (past_l2 ? launch_permute<16, true>(p, row_bytes, grid, smem, st)
                            : launch_permute<16, false>(p, row_bytes, grid, smem, st))
        : units(4) ? launch_permute<4, false>(p, row_bytes, grid, smem, st)
                   : launch_permute<2, false>(p, row_bytes, grid, smem, st);
    if (e != cudaSuccess) return cuda_fail(e, "permute launch");
    return QMOE_OK;
}

qmoe_status moe_combine(int ytype, const void* y, int64_t n_rows, int64_t cols, int64_t ldy,
                        const int32_t* pos, const float* topk_w, int64_t n_tokens, int32_t top_k,
                        int otype, const void* residual, void* out, int64_t ldo, void* stream) {
    clear_error();
    const char* fn = "moe_combine";
    if (qmoe_status s = combine_check(fn, ytype, y, n_rows, cols, ldy, pos, topk_w, n_tokens, top_k,
                                      otype, ldo))
        return s;
    if (n_tokens == 0) return QMOE_OK;
    const int os = float_size(otype);
    if (!out || !aligned(out, os) || !aligned(residual, os))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: out null, or out or residual not aligned to their elements", fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    steps::CombineParams p = {};
    p.y = y;
    p.n_rows = n_rows;
    p.ldy = ldy;
    p.cols = static_cast<int>(cols);
    p.pos = pos;
    p.w = topk_w;
    p.k = top_k;
    p.residual = residual;
    p.out = out;
    p.ldo = ldo;
    return run_combine(p, ytype, otype, n_tokens, static_cast<cudaStream_t>(stream));
}

qmoe_status moe_combine_backward(int ytype, const void* y, int64_t n_rows, int64_t cols,
                                 int64_t ldy, const int32_t* pos, const float* topk_w,
                                 int64_t n_tokens, int32_t top_k, int otype, const void* grad_out,
                                 int64_t ldo, void* grad_y, int64_t ldg, float* grad_w,
                                 void* stream) {
    clear_error();
    const char* fn = "moe_combine_backward";
    if (!grad_y && !grad_w)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: grad_y and grad_w are both null", fn);
    // (without grad_w the rows are not read and y may be null)
    if (qmoe_status s = combine_check(fn, ytype, grad_w ? y : grad_y, n_rows, cols, ldy, pos,
                                      topk_w, n_tokens, top_k, otype, ldo))
        return s;
    if (grad_y && ldg < cols)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: ldg=%lld must be >= cols=%lld", fn,
                    (long long)ldg, (long long)cols);
    if (n_tokens == 0) return QMOE_OK;
    if (!grad_out || !aligned(grad_out, float_size(otype)) || !aligned(grad_y, float_size(ytype)) ||
        !aligned(grad_w, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: grad_out null, or a gradient not aligned to its elements", fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    steps::CombineParams p = {};
    p.y = grad_w ? y : nullptr;
    p.n_rows = n_rows;
    p.ldy = grad_w ? ldy : 0;
    p.cols = static_cast<int>(cols);
    p.pos = pos;
    p.w = topk_w;
    p.k = top_k;
    p.ldo = ldo;
    p.grad_out = grad_out;
    p.grad_y = grad_y;
    p.ldg = grad_y ? ldg : 0;
    p.grad_w = grad_w;
    return run_combine(p, ytype, otype, n_tokens, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
