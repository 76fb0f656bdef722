// f8.cu — entry points of the e4m3 block-scaled and expert-grouped products:
// argument validation, launch planning and launches of the kernels of
// gmm.cuh and f8moe.cuh.  See include/qmoe.h for the contract of every
// function.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "../../include/qmoe.h"
#include "host.cuh"
#include "gmm.cuh"
#include "gmm_pair.cuh"
#include "f8moe.cuh"

namespace qmoe {

static int type_size(int t) {
    switch (t) {
    case QMOE_F32: return 4;
    case QMOE_BF16: case QMOE_F16: return 2;
    case QMOE_E4M3: return 1;
    default: return 0;
    }
}
static bool float_type(int t) { return t == QMOE_F32 || t == QMOE_BF16 || t == QMOE_F16; }
static int out_type(int t) {
    return t == QMOE_BF16 ? gmm::OUT_BF16 : t == QMOE_F16 ? gmm::OUT_F16 : gmm::OUT_F32;
}

constexpr int64_t MAX_COLS = 1 << 20;    // K of a product, columns of a quantised row
constexpr int64_t MAX_ROWS = 0x7fffff00; // token rows and weight rows
constexpr int MAX_GROUPS = 1024;
constexpr int MAX_F8_EXPERTS = 256;
constexpr int MAX_F8_TOPK = 16;  // the kernels hold a token's slots in 16 lanes

// ------------------------------------------------------------ tensor maps
// [outer][rows][inner] elements of `size` bytes, 128-byte swizzled boxes of
// one 128-byte run of K by box_rows rows.
static qmoe_status operand_map(CUtensorMap* m, const void* base, int size, bool bf16,
                               int64_t inner, int64_t rows, int64_t outer, int64_t row_stride,
                               int box_rows) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return fail(QMOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(outer)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride) * size,
                                   static_cast<cuuint64_t>(row_stride) * size * rows};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(gmm::KBLK / size),
                               static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    const CUtensorMapDataType dt = size == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : bf16    ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUresult r = fn(m, dt, outer > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box,
                          estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(QMOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return QMOE_OK;
}

// ------------------------------------------------------- grouped products
struct Gmm {
    int type;           // QMOE_E4M3, QMOE_BF16, QMOE_F16
    const void* W;      // [E][N][K]
    const void* W2;     // second stack (SwiGLU form) or null
    const void* x;      // [M][K], rows ldx apart
    int64_t K, ldx;
    gmm::Params p;
};

// Launches kernel `kern` of configuration C; `shaped`: as clusters of `ranks`
// CTAs (the pair kernel has its cluster shape in its code).
template <class C, class Kern>
static qmoe_status launch_gmm(Kern kern, int threads, bool shaped, const Gmm& g, int ranks,
                              int clusters, const DevInfo& d, cudaStream_t st) {
    const int smem = C::smem(g.p.E);
    constexpr int most = C::smem(C::GU ? MAX_F8_EXPERTS : MAX_GROUPS);
    static_assert(most + 512 <= 232448, "shared memory of one CTA, static arrays included");
    static std::atomic<int> configured[64];
    if (smem > configured[d.dev].load()) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             most);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(grouped product)");
        configured[d.dev].store(most);
    }
    const int size = type_size(g.type);
    const bool bf16 = g.type == QMOE_BF16;
    CUtensorMap tw, tw2, tx;
    if (qmoe_status s = operand_map(&tw, g.W, size, bf16, g.K, g.p.N, g.p.E, g.K, gmm::TILE_W))
        return s;
    tw2 = tw;
    if (g.W2)
        if (qmoe_status s = operand_map(&tw2, g.W2, size, bf16, g.K, g.p.N, g.p.E, g.K,
                                        gmm::TILE_W))
            return s;
    if (qmoe_status s = operand_map(&tx, g.x, size, bf16, g.K, g.p.M, 0, g.ldx, C::BOX)) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * ranks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
    cfg.numAttrs = shaped ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, g.p, tw, tw2, tx);
    if (e != cudaSuccess) return cuda_fail(e, "grouped product launch");
    return QMOE_OK;
}

// The kernel for few rows per group.  Fewer tiles than SMs: clusters of as many
// CTAs as the SMs have room for share a tile's K range; else one CTA per SM
// takes tile after tile.
template <class C>
static qmoe_status launch_few(const Gmm& g, const DevInfo& d, cudaStream_t st) {
    const int64_t tiles = gmm::max_tiles(g.p.M, g.p.E, C::NT, g.p.nb);
    int ranks = 1;
    if (tiles < d.sms) {
        // (a power of two: clusters of three left SMs of a GPC idle and took a
        // second wave: 48 tiles on 144 CTAs 19 us, on 96 CTAs half of it)
        while (ranks < gmm::MAX_RANKS && 2 * ranks * tiles <= d.sms && 2 * ranks <= g.p.kb)
            ranks *= 2;
    }
    const int clusters = static_cast<int>(tiles < d.sms ? tiles : d.sms);
    return launch_gmm<C>(gmm::gmm_kernel<C>, gmm::THREADS, true, g, ranks, clusters, d, st);
}

// One CTA pair per two SMs, or as many as there can be tiles.
template <class C>
static qmoe_status launch_pairs(const Gmm& g, const DevInfo& d, cudaStream_t st) {
    const int64_t tiles = gmm::max_tiles(g.p.M, g.p.E, C::NT, (g.p.nb + 1) / 2);
    const int pairs = static_cast<int>(tiles < d.sms / 2 ? tiles : d.sms / 2);
    return launch_gmm<C>(gmm::gmm_pair_kernel<C>, C::THREADS, false, g, 2, pairs, d, st);
}

static qmoe_status run_gmm(Gmm g, const DevInfo& d, cudaStream_t st) {
    const int size = type_size(g.type);
    g.p.kb = static_cast<int>((g.K * size + gmm::KBLK - 1) / gmm::KBLK);
    g.p.nb = (g.p.N + gmm::TILE_W - 1) / gmm::TILE_W;
    g.p.err = d.err;
    g.p.vec_out = g.p.out != gmm::OUT_F32 && aligned(g.p.y, 16) && g.p.ldy % 8 == 0;
    // D f32 (bit 4); 16-bit operands: 0 f16, 1 bf16 (bits 7-9 and 10-12);
    // 8-bit operands: 0 e4m3; M / 16 from bit 24
    const uint32_t fmt = g.type == QMOE_BF16 ? 1u : 0u;
    g.p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) |
                (static_cast<uint32_t>(gmm::TILE_W >> 4) << 24);
    const bool f8 = g.type == QMOE_E4M3;
    const int nt = gmm::token_tile(g.p.M, g.p.E, g.p.offsets != nullptr, g.p.nb, f8,
                                   g.W2 != nullptr, d.sms);
    if (nt == gmm::FEW_ROWS) {
        if (g.W2) return launch_few<gmm::Cfg<true, 5, true>>(g, d, st);
        return f8 ? launch_few<gmm::Cfg<true, 8, false>>(g, d, st)
                  : launch_few<gmm::Cfg<false, 8, false>>(g, d, st);
    }
    g.p.idesc += static_cast<uint32_t>(gmm::TILE_W >> 4) << 24;  // M = 256
    if (g.W2) return launch_pairs<gmm::PairCfg<true, 96, 5, true, 3>>(g, d, st);
    if (f8)
        return nt == 128 ? launch_pairs<gmm::PairCfg<true, 128, 7, false, 4>>(g, d, st)
                         : launch_pairs<gmm::PairCfg<true, 192, 6, false, 3>>(g, d, st);
    return nt == 128 ? launch_pairs<gmm::PairCfg<false, 128, 7, false, 4>>(g, d, st)
                     : launch_pairs<gmm::PairCfg<false, 256, 5, false, 3>>(g, d, st);
}

// --------------------------------------------------------------- quantise
template <class T, bool VEC, int RUN>
static cudaError_t launch_quantize_run(f8::QuantParams q, cudaStream_t st) {
    q.nrun = (q.nblk + RUN - 1) / RUN;
    const int64_t items = q.rows * q.nrun;
    const unsigned grid = static_cast<unsigned>((items + f8::Q_THREADS / 16 - 1) /
                                                (f8::Q_THREADS / 16));
    return launch_pdl(f8::quantize_kernel<T, VEC, RUN>, dim3(grid), dim3(f8::Q_THREADS), 0, st, q);
}
template <class T>
static cudaError_t launch_quantize(const f8::QuantParams& q, int sms, cudaStream_t st) {
    const bool vec = q.cols % 8 == 0 && (q.ldx * sizeof(T)) % 16 == 0 && aligned(q.x, 16) &&
                     aligned(q.q, 8);
    // runs of four blocks once they fill the GPU's threads
    const bool many = q.rows * q.nblk >= static_cast<int64_t>(sms) * (2048 / 16) * 2;
    return vec ? (many ? launch_quantize_run<T, true, 4>(q, st)
                       : launch_quantize_run<T, true, 1>(q, st))
               : launch_quantize_run<T, false, 1>(q, st);
}
template <class T>
static cudaError_t launch_group_quantize(const f8::QuantParams& q, const int32_t* idx, int P, int E,
                                         int32_t* offsets, int32_t* pos, cudaStream_t st) {
    return launch_pdl(f8::group_quantize_kernel<T>, dim3(static_cast<unsigned>(q.rows)),
                      dim3(f8::Q_THREADS), 0, st, q, idx, P, E, offsets, pos);
}
static qmoe_status run_quantize(int type, const f8::QuantParams& q, int sms, cudaStream_t st) {
    const cudaError_t e = type == QMOE_F32    ? launch_quantize<float>(q, sms, st)
                          : type == QMOE_BF16 ? launch_quantize<__nv_bfloat16>(q, sms, st)
                                              : launch_quantize<__half>(q, sms, st);
    if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
    return QMOE_OK;
}

// ------------------------------------------------------------- MoE layer
struct MoeWs {
    size_t offsets, pos, xq, xs, aq, as, y, total;
};
static MoeWs moe_f8_layout(const qmoe_moe_shape& s) {
    const size_t P = static_cast<size_t>(s.n_tokens) * s.top_k, E = s.num_experts, H = s.hidden,
                 F = s.expert_dim;
    auto al = [](size_t v) { return (v + 255) / 256 * 256; };
    MoeWs w;
    size_t o = 0;
    w.offsets = o; o += al((E + 1) * 4);
    w.pos = o;     o += al(P * 4);
    w.xq = o;      o += al(P * H);
    w.xs = o;      o += al(P * (H / F8_BLOCK) * 4);
    w.aq = o;      o += al(P * F);
    w.as = o;      o += al(P * (F / F8_BLOCK) * 4);
    w.y = o;       o += al(P * H * 4);
    w.total = o;
    return w;
}

// Shape rules of moe_experts_f8 (also behind its workspace size).
static qmoe_status moe_f8_shape(const qmoe_moe_shape* s) {
    const char* fn = "moe_experts_f8";
    if (!s) return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null shape", fn);
    if (s->hidden <= 0 || s->expert_dim <= 0 || s->num_experts <= 0 || s->top_k <= 0 ||
        s->n_tokens < 0)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: incomplete MoE shape (hidden=%d expert_dim=%d num_experts=%d top_k=%d "
                    "n_tokens=%d)",
                    fn, s->hidden, s->expert_dim, s->num_experts, s->top_k, s->n_tokens);
    if (s->route_flags)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: route_flags=0x%x must be 0 (the routes are given)", fn,
                    static_cast<unsigned>(s->route_flags));
    if (s->gate_qtype != QMOE_E4M3 || s->up_qtype != QMOE_E4M3 || s->down_qtype != QMOE_E4M3)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: gate, up and down must be E4M3 (%d %d %d)", fn,
                    s->gate_qtype, s->up_qtype, s->down_qtype);
    if (s->num_experts > MAX_F8_EXPERTS || s->top_k > MAX_F8_TOPK)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: num_experts=%d > %d or top_k=%d > %d", fn,
                    s->num_experts, MAX_F8_EXPERTS, s->top_k, MAX_F8_TOPK);
    if (s->hidden % F8_BLOCK || s->expert_dim % F8_BLOCK)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: hidden=%d and expert_dim=%d must be multiples of %d",
                    fn, s->hidden, s->expert_dim, F8_BLOCK);
    if (s->hidden > MAX_COLS || s->expert_dim > MAX_COLS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: hidden or expert_dim exceeds %lld", fn,
                    (long long)MAX_COLS);
    if (static_cast<int64_t>(s->n_tokens) * s->top_k > MAX_ROWS / 64)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: n_tokens * top_k exceeds %lld", fn,
                    (long long)(MAX_ROWS / 64));
    return QMOE_OK;
}

template <class T, class Y>
static cudaError_t launch_combine(const void* y, const int32_t* pos, const float* w,
                                  const void* residual, void* out, int T_, int H, int k,
                                  cudaStream_t st) {
    const int per = f8::C_THREADS * 8;
    return launch_pdl(f8::combine_kernel<T, Y>, dim3(T_, (H + per - 1) / per),
                      dim3(f8::C_THREADS), 0, st, static_cast<const Y*>(y), pos, w,
                      static_cast<const T*>(residual), static_cast<T*>(out), H, k);
}

// The group kernel: a CTA for every 512 pairs, up to a cluster of eight.
static cudaError_t launch_group(const int32_t* idx, int P, int E, int32_t* offsets, int32_t* pos,
                                cudaStream_t st) {
    int ranks = 1;
    while (ranks < f8::G_CLUSTER && ranks * 512 < P) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ranks));
    cfg.blockDim = dim3(f8::G_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(f8::G_WARPS + 1) * E * 4;
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
    return cudaLaunchKernelEx(&cfg, f8::group_kernel, idx, P, E, offsets, pos);
}

}  // namespace qmoe

using namespace qmoe;

// ====================================================================== C ABI
extern "C" {

qmoe_status f8_quantize(int xtype, const void* x, int64_t rows, int64_t cols, int64_t ldx, void* q,
                        float* scale, void* stream) {
    clear_error();
    const char* fn = "f8_quantize";
    if (!float_type(xtype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: x type %d is not F32, BF16 or F16", fn, xtype);
    if (rows < 0 || cols <= 0 || ldx < cols)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: rows=%lld >= 0, cols=%lld >= 1 and ldx=%lld >= cols are needed", fn,
                    (long long)rows, (long long)cols, (long long)ldx);
    if (cols > MAX_COLS || rows > MAX_ROWS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: cols=%lld > %lld or rows=%lld > %lld", fn,
                    (long long)cols, (long long)MAX_COLS, (long long)rows, (long long)MAX_ROWS);
    if (rows == 0) return QMOE_OK;
    if (!x || !q || !scale) return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer", fn);
    if (!aligned(x, type_size(xtype)) || !aligned(scale, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: x and scale must be aligned to their elements",
                    fn);
    f8::QuantParams p = {};
    p.x = x;
    p.ldx = ldx;
    p.q = static_cast<uint8_t*>(q);
    p.s = scale;
    p.rows = rows;
    p.cols = static_cast<int>(cols);
    p.nblk = static_cast<int>((cols + F8_BLOCK - 1) / F8_BLOCK);
    if (rows * p.nblk > (int64_t{1} << 34))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: rows=%lld x cols=%lld has more than 2^34 blocks", fn,
                    (long long)rows, (long long)cols);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    return run_quantize(xtype, p, d->sms, static_cast<cudaStream_t>(stream));
}

// Checks shared by f8_mm and mm_grouped.
static qmoe_status mm_check(const char* fn, int wtype, const void* W, const float* w_scale,
                            int64_t rows, int64_t cols, const void* x, const float* x_scale,
                            int64_t n_rows, int64_t ldx, int ytype, const void* y, int64_t ldy) {
    const int size = type_size(wtype);
    if (!float_type(ytype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: y type %d is not F32, BF16 or F16", fn, ytype);
    if (rows <= 0 || cols <= 0 || n_rows < 0 || ldx < cols || ldy < rows)
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: rows=%lld, cols=%lld >= 1, n=%lld >= 0, ldx=%lld >= cols and ldy=%lld >= "
                    "rows are needed",
                    fn, (long long)rows, (long long)cols, (long long)n_rows, (long long)ldx,
                    (long long)ldy);
    if (rows > MAX_ROWS || n_rows > MAX_ROWS || cols > MAX_COLS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: rows=%lld, n=%lld or cols=%lld is too large", fn,
                    (long long)rows, (long long)n_rows, (long long)cols);
    if ((cols * size) % 16 || (ldx * size) % 16)
        return fail(QMOE_ERR_UNSUPPORTED,
                    "%s: cols=%lld and ldx=%lld must be multiples of %d (16 bytes)", fn,
                    (long long)cols, (long long)ldx, 16 / size);
    if (n_rows == 0) return QMOE_OK;
    if (!W || !x || !y) return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer (W, x or y)", fn);
    if (wtype == QMOE_E4M3 && (!w_scale || !x_scale))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: E4M3 operands need w_scale and x_scale", fn);
    if (wtype != QMOE_E4M3 && (w_scale || x_scale))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: scales are for E4M3 operands only", fn);
    if (!aligned(W, 16) || !aligned(x, 16) || !aligned(y, type_size(ytype)) ||
        !aligned(w_scale, 4) || !aligned(x_scale, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT,
                    "%s: W and x must be 16-byte aligned, y and the scales aligned to their "
                    "elements",
                    fn);
    return QMOE_OK;
}

qmoe_status f8_mm(const void* W, const float* w_scale, int64_t rows, int64_t cols, const void* x,
                  const float* x_scale, int64_t n_tokens, int64_t ldx, int ytype, void* y,
                  int64_t ldy, void* stream) {
    clear_error();
    if (qmoe_status s = mm_check("f8_mm", QMOE_E4M3, W, w_scale, rows, cols, x, x_scale, n_tokens,
                                 ldx, ytype, y, ldy))
        return s;
    if (n_tokens == 0) return QMOE_OK;
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    Gmm g = {};
    g.type = QMOE_E4M3;
    g.W = W;
    g.x = x;
    g.K = cols;
    g.ldx = ldx;
    g.p.xs = x_scale;
    g.p.ws = w_scale;
    g.p.y = y;
    g.p.ldy = ldy;
    g.p.M = static_cast<int>(n_tokens);
    g.p.N = static_cast<int>(rows);
    g.p.E = 1;
    g.p.out = out_type(ytype);
    return run_gmm(g, *d, static_cast<cudaStream_t>(stream));
}

qmoe_status mm_grouped(int wtype, const void* W, const float* w_scale, int32_t num_groups,
                       int64_t rows, int64_t cols, const void* x, const float* x_scale,
                       int64_t n_rows, int64_t ldx, const int32_t* offsets, int ytype, void* y,
                       int64_t ldy, void* stream) {
    clear_error();
    const char* fn = "mm_grouped";
    if (wtype != QMOE_E4M3 && wtype != QMOE_BF16 && wtype != QMOE_F16)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: type %d is not E4M3, BF16 or F16", fn, wtype);
    if (num_groups <= 0)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: num_groups=%d must be >= 1", fn, num_groups);
    if (num_groups > MAX_GROUPS)
        return fail(QMOE_ERR_UNSUPPORTED, "%s: num_groups=%d exceeds %d", fn, num_groups,
                    MAX_GROUPS);
    if (qmoe_status s = mm_check(fn, wtype, W, w_scale, rows, cols, x, x_scale, n_rows, ldx, ytype,
                                 y, ldy))
        return s;
    if (n_rows == 0) return QMOE_OK;
    if (!offsets || !aligned(offsets, 4))
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: offsets null or not 4-byte aligned", fn);
    DevInfo* d = nullptr;
    if (qmoe_status s = device_info(&d)) return s;
    Gmm g = {};
    g.type = wtype;
    g.W = W;
    g.x = x;
    g.K = cols;
    g.ldx = ldx;
    g.p.offsets = offsets;
    g.p.xs = x_scale;
    g.p.ws = w_scale;
    g.p.y = y;
    g.p.ldy = ldy;
    g.p.M = static_cast<int>(n_rows);
    g.p.N = static_cast<int>(rows);
    g.p.E = num_groups;
    g.p.out = out_type(ytype);
    return run_gmm(g, *d, static_cast<cudaStream_t>(stream));
}

size_t moe_experts_f8_workspace_size(const qmoe_moe_shape* shape) {
    clear_error();
    if (moe_f8_shape(shape)) return 0;
    return moe_f8_layout(*shape).total;
}

qmoe_status moe_experts_f8(const void* gate_stack, const float* gate_scale, const void* up_stack,
                           const float* up_scale, const void* down_stack, const float* down_scale,
                           const qmoe_moe_shape* shape, int xtype, const void* x,
                           const int32_t* topk_idx, const float* topk_w, const void* residual,
                           void* out, void* ws, size_t ws_bytes, void* stream) {
    clear_error();
    const char* fn = "moe_experts_f8";
    if (qmoe_status r = moe_f8_shape(shape)) return r;
    const qmoe_moe_shape s = *shape;
    if (!float_type(xtype))
        return fail(QMOE_ERR_UNSUPPORTED, "%s: x type %d is not F32, BF16 or F16", fn, xtype);
    if (s.n_tokens == 0) return QMOE_OK;
    if (!gate_stack || !gate_scale || !up_stack || !up_scale || !down_stack || !down_scale || !x ||
        !topk_idx || !topk_w || !out || !ws)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: null pointer", fn);
    const MoeWs L = moe_f8_layout(s);
    if (ws_bytes < L.total)
        return fail(QMOE_ERR_INVALID_ARGUMENT, "%s: workspace %zu < %zu bytes", fn, ws_bytes,
                    L.total);
    for (const void* q : {gate_stack, up_stack, down_stack, x, residual,
                          static_cast<const void*>(out), static_cast<const void*>(ws)})
        if (!aligned(q, 16))
            return fail(QMOE_ERR_INVALID_ARGUMENT,
                        "%s: stacks, x, residual, out and ws must be 16-byte aligned", fn);
    for (const void* q : {static_cast<const void*>(gate_scale), static_cast<const void*>(up_scale),
                          static_cast<const void*>(down_scale),
                          static_cast<const void*>(topk_idx), static_cast<const void*>(topk_w)})
        if (!aligned(q, 4))
            return fail(QMOE_ERR_INVALID_ARGUMENT,
                        "%s: scales, topk_idx and topk_w must be 4-byte aligned", fn);
    DevInfo* d = nullptr;
    if (qmoe_status r = device_info(&d)) return r;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    int32_t* offsets = reinterpret_cast<int32_t*>(w + L.offsets);
    int32_t* pos = reinterpret_cast<int32_t*>(w + L.pos);
    void* y = w + L.y;
    const int T = s.n_tokens, k = s.top_k, H = s.hidden, F = s.expert_dim, E = s.num_experts;
    const int P = T * k;

    f8::QuantParams q = {};
    q.x = x;
    q.ldx = H;
    q.q = w + L.xq;
    q.s = reinterpret_cast<float*>(w + L.xs);
    q.pos = pos;
    q.k = k;
    q.rows = T;
    q.cols = H;
    q.nblk = H / F8_BLOCK;
    cudaError_t e;
    if (P <= f8::GQ_PAIRS) {
        e = xtype == QMOE_F32 ? launch_group_quantize<float>(q, topk_idx, P, E, offsets, pos, st)
            : xtype == QMOE_BF16
                ? launch_group_quantize<__nv_bfloat16>(q, topk_idx, P, E, offsets, pos, st)
                : launch_group_quantize<__half>(q, topk_idx, P, E, offsets, pos, st);
        if (e != cudaSuccess) return cuda_fail(e, "group and quantize launch");
    } else {
        e = launch_group(topk_idx, P, E, offsets, pos, st);
        if (e != cudaSuccess) return cuda_fail(e, "group launch");
        if (qmoe_status r = run_quantize(xtype, q, d->sms, st)) return r;
    }

    Gmm g = {};
    g.type = QMOE_E4M3;
    g.W = gate_stack;
    g.W2 = up_stack;
    g.x = q.q;
    g.K = H;
    g.ldx = H;
    g.p.offsets = offsets;
    g.p.xs = q.s;
    g.p.ws = gate_scale;
    g.p.ws2 = up_scale;
    g.p.aq = w + L.aq;
    g.p.as = reinterpret_cast<float*>(w + L.as);
    g.p.M = P;
    g.p.N = F;
    g.p.E = E;
    if (qmoe_status r = run_gmm(g, *d, st)) return r;

    Gmm h = {};
    h.type = QMOE_E4M3;
    h.W = down_stack;
    h.x = g.p.aq;
    h.K = F;
    h.ldx = F;
    h.p.offsets = offsets;
    h.p.xs = g.p.as;
    h.p.ws = down_scale;
    h.p.y = y;
    h.p.ldy = H;
    h.p.M = P;
    h.p.N = H;
    h.p.E = E;
    h.p.out = xtype == QMOE_BF16 ? gmm::OUT_BF16 : gmm::OUT_F32;
    if (qmoe_status r = run_gmm(h, *d, st)) return r;

    e = xtype == QMOE_F32 ? launch_combine<float, float>(y, pos, topk_w, residual, out, T, H, k, st)
        : xtype == QMOE_BF16
            ? launch_combine<__nv_bfloat16, __nv_bfloat16>(y, pos, topk_w, residual, out, T, H, k,
                                                           st)
            : launch_combine<__half, float>(y, pos, topk_w, residual, out, T, H, k, st);
    if (e != cudaSuccess) return cuda_fail(e, "combine launch");
    return QMOE_OK;
}

}  // extern "C"
