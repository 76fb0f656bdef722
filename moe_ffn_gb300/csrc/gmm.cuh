// gmm.cuh — matrix products grouped by expert on the 5th-generation tensor
// cores: y[r] = x[r] W_e^T for the rows r of group e, W an [E][N][K] stack of
// row-major matrices, in f16, bf16, or e4m3 with f32 scales (x: one per row
// and 128 columns; W: one per 128 x 128 block).  One matrix is the case of
// one group.
//
// Orientation: the weight rows are the MMA's M side (128 of them = the 128
// TMEM lanes), the token rows its N side.  A group of n rows then costs
// about n / 16 of an N side in steps of 16, down to one token, with the
// weights streamed once per token tile; and the epilogue's stores run along
// a row of y.
//
// Scales.  With sx[r][b] and sw[e][n/128][b] for k-block b,
//   y[r][n] = sum_b sx sw sum_{k in b} xq Wq.
// The tensor core forms the inner sum of one k-block exactly as products
// and in f32 as sums; the epilogue warps then add (sx sw) * partial to f32
// registers while the tensor core works on the next blocks.  f16/bf16 products
// accumulate in TMEM over the whole of K.
//
// This file holds the parts all forms share and the kernel for few rows per
// group (gmm_kernel): bound by streaming the weights, so its tiles are small
// (128 weight rows, 32 tokens) and, where there are fewer tiles than SMs, the
// CTAs of a cluster share a tile's K range and add their parts through
// distributed shared memory, in rank order.  gmm_pair.cuh has the kernel for
// many rows.
//
// Measured: 1 x 4096 x 4096 e4m3 6.6 us (fixed latency: about 2,500 clocks to
// the first copy, 1,300 for its data, 3,000 from the last MMA to the end); eight
// bf16 experts of one row, 768 x 2048: 8.6 us, 2.9 TB/s; 128 rows in 64 groups,
// 2048 x 2048 bf16: 81 us, 6.7 TB/s.
//
// Warp roles (384 threads): warp 0 loads (TMA), warp 1 issues the MMAs, warp 2
// stages the scale products (warp 3 has no part: the epilogue's warps start at a
// multiple of four), warps 4-11 are the epilogue: warp w reads TMEM lanes
// 32 (w % 4) .. +31, and the two groups of four warps take sixteen columns each.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f8.cuh"
#include "gmm_tiles.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace qmoe {
namespace gmm {

constexpr int TILE_W = 128;    // weight rows per tile
constexpr int KBLK = 128;      // bytes of K per stage and operand row
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int SC_BLK = 4;      // k-blocks of scales staged at a time
constexpr int SC_RING = 3;     // such stages

enum OutType : int { OUT_F32 = 0, OUT_BF16 = 1, OUT_F16 = 2 };

struct Params {
    const int32_t* offsets;  // [E+1] rows of each group, or null: one group of all rows
    const float* xs;         // [M][kb] scales of x (e4m3)
    const float* ws;         // [E][nb][kb] scales of W (gate)
    const float* ws2;        // [E][nb][kb] scales of the second matrix (up)
    void* y;                 // [M][ldy]
    uint8_t* aq;             // SwiGLU form: [M][N] e4m3 activations
    float* as;               //              [M][nb] their scales
    int64_t ldy;
    int M, N, E;
    int kb;                  // 128-byte blocks of K
    int nb;                  // 128-row tiles of W
    int out;                 // OutType
    int vec_out;             // y is 16-bit with 16-byte aligned rows
    uint32_t idesc;          // instruction descriptor without N
    DevCtl* err;
};

// Configuration of one instantiation of the kernel for few rows.
//   F8     e4m3 operands with scales (else 16-bit)
//   NST    pipeline stages
//   GU     two weight stacks (gate, up) and the SwiGLU + e4m3 epilogue
template <bool F8_, int NST_, bool GU_>
struct Cfg {
    static constexpr bool F8 = F8_, GU = GU_;
    static constexpr int NT = FEW_ROWS, NST = NST_;  // token tile
    static constexpr int NA = GU ? 2 : 1;
    static constexpr int BOX = NT;  // a stage's token rows are one TMA box
    static constexpr int A_BYTES = TILE_W * KBLK;
    static constexpr int STAGE = NA * A_BYTES + NT * KBLK;
    static constexpr int CH = 16;  // columns per epilogue warp
    static constexpr int NBUF = 4;                 // accumulator buffers
    static constexpr int TM_BUF = NA * NT;         // TMEM columns per buffer
    static constexpr int TM_COLS = NBUF * TM_BUF;
    static constexpr int SC_STAGE = SC_BLK * NA * NT;  // floats
    // byte offsets in shared memory
    static constexpr int O_SC = NST * STAGE;
    static constexpr int O_PART = O_SC + (F8 ? SC_RING * SC_STAGE * 4 : 0);
    static constexpr int O_AMAX = O_PART + NA * NT * TILE_W * 4;
    static constexpr int O_BAR = O_AMAX + (GU ? 2 * 4 * NT * 4 : 0);
    static constexpr int N_BAR = 2 * NST + 2 * SC_RING + 2 * NBUF + 1 + (GU ? 2 : 0);
    static constexpr int O_TAB = O_BAR + (N_BAR + 1) * 8;
    // tables: first row, end row and first tile of each group, total last
    static constexpr int smem(int E) { return 1024 + O_TAB + (3 * E + 4) * 4; }
    static_assert((TM_COLS & (TM_COLS - 1)) == 0 && TM_COLS <= 512, "TMEM columns");
};
constexpr int MAX_RANKS = 8;  // CTAs that may share a tile

// a += v * s on pairs (one packed FMA), v as bits.
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, float s0,
                                     float s1) {
    asm("{\n\t.reg .b64 a, v, s;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %5};\n\t"
        "fma.rn.f32x2 a, v, s, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "r"(v0), "r"(v1), "f"(s0), "f"(s1));
}

__device__ __forceinline__ void store_out(void* y, int64_t i, int type, float v) {
    if (type == OUT_BF16)
        static_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
    else if (type == OUT_F16)
        static_cast<__half*>(y)[i] = __float2half_rn(v);
    else
        static_cast<float*>(y)[i] = v;
}

// silu(g) u.  With e = exp(-|g|) <= 1 the quotient's divisor lies in [1, 2]: no
// overflow for any g, where 1 + exp(-g) passed the divisor's range of the fast
// division at g = -87.3 and gave 0.  Roundings: e 2 ulp and 1 + e half (at most
// 1.5 in the divisor), g e half, the fast division 2, the product half: within 7
// ulp or 2^-20 (below g = -87 e is subnormal and its last bits go).  The fast
// exponential is off by up to 1.2 |g| ulp.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.0f + e) * u;
}

// The cluster's values at this CTA's address `src`, added in rank order; all
// loads are issued before the first sum.
__device__ __forceinline__ float cluster_sum(const float* src, int ranks) {
    float v[MAX_RANKS];
#pragma unroll
    for (int q = 0; q < MAX_RANKS; ++q)
        v[q] = q < ranks ? cluster_ld_f32(src, static_cast<uint32_t>(q)) : 0.f;
    float s = v[0];
#pragma unroll
    for (int q = 1; q < MAX_RANKS; ++q)
        if (q < ranks) s += v[q];
    return s;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The groups' tables, by the whole CTA (ends with a barrier): rows [lo, hi) of
// each group and the tiles before it, the total last.  If any group's offsets
// decrease or leave [0, M] the total is 0 and the call computes nothing: clamped
// groups may overlap, so two would write the same rows, and their tiles may be
// more than an int counts.  A thread per group; the time is one load latency and
// one scan.
__device__ __forceinline__ void build_tables(const Params& p, int nt, int nb, int* t_lo,
                                             int* t_hi, int* t_pre) {
    __shared__ int wsum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int total = 0, bad = 0;
    for (int e0 = 0; e0 < p.E; e0 += blockDim.x) {
        const int e = e0 + tid;
        int n = 0;
        if (e < p.E) {
            int lo = 0, hi = p.M;
            if (p.offsets &&
                !group_rows(__ldcg(p.offsets + e), __ldcg(p.offsets + e + 1), p.M, &lo, &hi)) {
                record_error(p.err, DEV_GMM_OFFSETS);
                bad = 1;
            }
            t_lo[e] = lo;
            t_hi[e] = hi;
            n = group_tiles(hi - lo, nt, nb);
        }
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        if (lane == 31) wsum[warp] = s;
        bad = __syncthreads_or(bad);
        const int nw = static_cast<int>(blockDim.x >> 5);
        int before = 0, all = 0;
        for (int w = 0; w < nw; ++w) {
            const int v = wsum[w];
            before += w < warp ? v : 0;
            all += v;
        }
        if (e < p.E) t_pre[e] = total + before + s - n;
        total += all;
        if (e0 + static_cast<int>(blockDim.x) < p.E) __syncthreads();  // wsum is used again
    }
    if (tid == 0) t_pre[p.E] = bad ? 0 : total;
    __syncthreads();
}

// k-blocks of a tile, counted from its end, whose stages no later load takes: the
// last NST steps of a CTA, `after` of them in tiles to come.  Such a stage is not
// handed back by a commit, so that every arrival of one is waited for: an arrival
// comes from the tensor core, no barrier between threads orders it, and the CTA's
// shared memory may be another launch's as soon as it ends.
template <int NST>
__device__ __forceinline__ int unreturned(int64_t after) {
    return after < NST ? NST - static_cast<int>(after) : 0;
}

template <class C>
__global__ void __launch_bounds__(THREADS, 1)
    gmm_kernel(const Params p, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_w2,
               const __grid_constant__ CUtensorMap tm_x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* ring = reinterpret_cast<float*>(base + C::O_SC);
    float* part = reinterpret_cast<float*>(base + C::O_PART);
    uint32_t* amax = reinterpret_cast<uint32_t*>(base + C::O_AMAX);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::O_BAR);
    uint64_t* full = bars;
    uint64_t* empty = full + C::NST;
    uint64_t* sc_full = empty + C::NST;
    uint64_t* sc_empty = sc_full + SC_RING;
    uint64_t* acc_full = sc_empty + SC_RING;
    uint64_t* acc_empty = acc_full + C::NBUF;
    uint64_t* mma_done = acc_empty + C::NBUF;
    uint64_t* am_full = mma_done + 1;  // [2] SwiGLU form: four warps' maxima are there
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BAR);
    int* t_lo = reinterpret_cast<int*>(base + C::O_TAB);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;  // [E+1]

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == 1) umma::tmem_alloc(tmem_slot, C::TM_COLS);
    if (tid == 0) {
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < SC_RING; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], EPI_WARPS);
        }
        for (int i = 0; i < C::NBUF; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], EPI_WARPS);
        }
        mbar_init(mma_done, 1);
        if constexpr (C::GU)
            for (int i = 0; i < 2; ++i) mbar_init(&am_full[i], 4);
        fence_barrier_init();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
        if constexpr (C::GU) prefetch_tensormap(&tm_w2);
    }
    // failure-path tests: this CTA's load warp issues nothing, so that every wait
    // that depends on it runs out
    const bool skip = __ldcg(&p.err->skip_arrive_cta) == static_cast<int>(blockIdx.x);
    // Every operand may be an earlier launch's output (weights quantised on
    // this stream too), so nothing is read before the dependency wait.
    pdl_wait();
    pdl_trigger();
    umma::fence_before_sync();
    build_tables(p, C::NT, p.nb, t_lo, t_hi, t_pre);
    umma::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = t_pre[p.E];

    // A cluster takes tiles first, first + step, ...; a cluster of more than one
    // CTA takes one tile, each of its CTAs a share of K.
    // The cluster size is a power of two.
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int lg = 31 - __clz(ranks);
    const int first = blockIdx.x >> lg;
    const int step = ranks > 1 ? max(tiles, 1) : gridDim.x;
    const int kbeg = (rank * p.kb) >> lg, kend = ((rank + 1) * p.kb) >> lg;
    Tile w0 = {};  // the first tile, for every role and the sum over the cluster
    if (first < tiles) w0 = tile_at_warp(first, C::NT, 16, t_lo, t_hi, t_pre, p.E);

    if (warp == 0) {
        // ---------------------------------------------------------- loads
        int it = 0, s = 0;
        uint32_t ph = 1;  // parity of the wait for a free stage
        bool ok = !skip;
        for (int t = first; t < tiles && ok; t += step) {
            const Tile w = t == first ? w0 : tile_at_warp(t, C::NT, 16, t_lo, t_hi, t_pre, p.E);
            for (int kb = kbeg; kb < kend; ++kb, ++it) {
                // (before any use of a stage the wait passes at once)
                if (!mbar_wait_spin(&empty[s], ph, p.err, DEV_GMM_TIMEOUT)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    uint8_t* st = base + s * C::STAGE;
                    mbar_arrive_expect_tx(&full[s], C::STAGE);
                    // x coordinates are multiples of 128 bytes; rows past the
                    // matrix or past x arrive as zeros
                    const int kx = C::F8 ? kb * KBLK : kb * (KBLK / 2);
                    tma_load_3d(st, &tm_w, kx, w.nbi * TILE_W, w.e, &full[s]);
                    if constexpr (C::GU)
                        tma_load_3d(st + C::A_BYTES, &tm_w2, kx, w.nbi * TILE_W, w.e, &full[s]);
                    tma_load_2d(st + C::NA * C::A_BYTES, &tm_x, kx, w.row0, &full[s]);
                }
                __syncwarp();
                if (++s == C::NST) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        // never leave with copies in flight
        for (int k = max(it - C::NST, 0); k < it; ++k)
            mbar_wait_spin(&full[k % C::NST], (k / C::NST) & 1, p.err, DEV_GMM_TIMEOUT);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        int s = 0;
        uint32_t ph = 0, ab = 0, aph = 1;  // stage and accumulator phases
        bool ok = true;
        const uint64_t da0 = umma::desc_sw128(smem_u32(base));
        const uint32_t hi = static_cast<uint32_t>(da0 >> 32), lo0 = static_cast<uint32_t>(da0);
        uint32_t lo = lo0;  // the stage's descriptor, low word
        for (int t = first; t < tiles && ok; t += step) {
            const Tile w = t == first ? w0 : tile_at_warp(t, C::NT, 16, t_lo, t_hi, t_pre, p.E);
            const uint32_t idesc = p.idesc | (static_cast<uint32_t>(w.np >> 3) << 17);
            const int ret = kend - unreturned<C::NST>(
                                       static_cast<int64_t>((tiles - 1 - t) / step) * (kend - kbeg));
#pragma unroll 1
            for (int kb = kbeg; kb < kend; ++kb) {
                const bool fresh = C::F8 || kb == kbeg;  // a new accumulator buffer
                const bool last = C::F8 || kb == kend - 1;
                // both waits tried before either is acted on
                bool r0 = mbar_try_wait(&full[s], ph), r1 = true;
                if (fresh) r1 = mbar_try_wait(&acc_empty[ab], aph);
                if (!r0) r0 = mbar_wait_spin(&full[s], ph, p.err, DEV_GMM_TIMEOUT);
                if (!r1) r1 = mbar_wait_spin(&acc_empty[ab], aph, p.err, DEV_GMM_TIMEOUT);
                if (!(r0 && r1)) {
                    ok = false;
                    break;
                }
                umma::fence_after_sync();
                if (elect_one()) {
                    const uint32_t d = tmem + ab * C::TM_BUF;
                    // 32 bytes of K further: the descriptors' address field + 2
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int a = 0; a < C::NA; ++a)
                            umma::mma_one<C::F8>(d + a * C::NT,
                                                 lo + a * (C::A_BYTES >> 4) + 2 * j,
                                                 lo + C::NA * (C::A_BYTES >> 4) + 2 * j, hi, idesc,
                                                 (!fresh || j > 0) ? 1u : 0u);
                    if (kb < ret) umma::commit(&empty[s]);
                    if (last) umma::commit(&acc_full[ab]);
                }
                __syncwarp();
                if (last && ++ab == C::NBUF) {
                    ab = 0;
                    aph ^= 1;
                }
                lo += C::STAGE >> 4;
                if (++s == C::NST) {
                    s = 0;
                    ph ^= 1;
                    lo = lo0;
                }
            }
        }
        // every MMA has finished before TMEM and the stages are given up
        if (elect_one()) umma::commit(mma_done);
        __syncwarp();
        mbar_wait_spin(mma_done, 0, p.err, DEV_GMM_TIMEOUT);
    } else if (warp == 2) {
        // --------------------------------------------------------- scales
        if constexpr (C::F8) {
            static_assert(C::NT == 32, "a token row per lane");
            // rows of scales are read four at a time where they are aligned
            const bool vec = (p.kb & 3) == 0 && (kbeg & 3) == 0 &&
                             (reinterpret_cast<uintptr_t>(p.xs) & 15) == 0;
            int ch = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = t == first ? w0 : tile_at_warp(t, C::NT, 16, t_lo, t_hi, t_pre, p.E);
                const int64_t wo = (static_cast<int64_t>(w.e) * p.nb + w.nbi) * p.kb;
                const float* xs = p.xs + (static_cast<int64_t>(w.row0) + lane) * p.kb;
                for (int k0 = kbeg; k0 < kend; k0 += SC_BLK, ++ch) {
                    float v[SC_BLK], g[C::NA][SC_BLK];
#pragma unroll
                    for (int b = 0; b < SC_BLK; ++b) {
                        g[0][b] = k0 + b < kend ? __ldcg(p.ws + wo + k0 + b) : 0.f;
                        if constexpr (C::GU)
                            g[1][b] = k0 + b < kend ? __ldcg(p.ws2 + wo + k0 + b) : 0.f;
                    }
                    if (vec && lane < w.nv && k0 + SC_BLK <= kend) {
                        const float4 q = __ldcg(reinterpret_cast<const float4*>(xs + k0));
                        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                    } else {
#pragma unroll
                        for (int b = 0; b < SC_BLK; ++b)
                            v[b] = lane < w.nv && k0 + b < kend ? __ldcg(xs + k0 + b) : 0.f;
                    }
                    const int s = ch % SC_RING, round = ch / SC_RING;
                    if (round > 0 && !mbar_wait_spin(&sc_empty[s], (round - 1) & 1, p.err,
                                                        DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    float* dst = ring + s * C::SC_STAGE;
#pragma unroll
                    for (int b = 0; b < SC_BLK; ++b)
#pragma unroll
                        for (int a = 0; a < C::NA; ++a)
                            dst[(b * C::NA + a) * C::NT + lane] = v[b] * g[a][b];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[s]);
                }
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------- epilogue
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const int col = half * C::CH;  // this warp's columns
        const uint32_t tm_run = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col;
        uint32_t ab = 0, aph = 0, cs = 0, cph = 0, par = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step, par ^= 1) {
            const Tile w = t == first ? w0 : tile_at_warp(t, C::NT, 16, t_lo, t_hi, t_pre, p.E);
            float acc[C::NA][C::CH];
#pragma unroll
            for (int a = 0; a < C::NA; ++a)
#pragma unroll
                for (int c = 0; c < C::CH; ++c) acc[a][c] = 0.f;
            const int periods = C::F8 ? kend - kbeg : 1;
            for (int k = 0; k < periods; ++k) {
                const int kk = k % SC_BLK;
                if (C::F8 && kk == 0)
                    ok = mbar_wait_spin(&sc_full[cs], cph, p.err, DEV_GMM_TIMEOUT);
                ok = ok && mbar_wait_spin(&acc_full[ab], aph, p.err, DEV_GMM_TIMEOUT);
                if (!ok) break;
                umma::fence_after_sync();
                if (col < w.np) {
                    uint32_t r[C::NA][C::CH];
#pragma unroll
                    for (int a = 0; a < C::NA; ++a)
                        umma::ld_32x32b_x16(tm_run + ab * C::TM_BUF + a * C::NT, r[a]);
#pragma unroll
                    for (int a = 0; a < C::NA; ++a) umma::wait_ld(r[a]);
                    if constexpr (C::F8) {
                        const float* sc =
                            ring + cs * C::SC_STAGE + kk * C::NA * C::NT + col;
#pragma unroll
                        for (int a = 0; a < C::NA; ++a)
#pragma unroll
                            for (int c = 0; c < C::CH; c += 4) {
                                const float4 s =
                                    *reinterpret_cast<const float4*>(sc + a * C::NT + c);
                                fma2(acc[a][c], acc[a][c + 1], r[a][c], r[a][c + 1], s.x, s.y);
                                fma2(acc[a][c + 2], acc[a][c + 3], r[a][c + 2], r[a][c + 3], s.z,
                                     s.w);
                            }
                    } else {
#pragma unroll
                        for (int c = 0; c < C::CH; ++c) acc[0][c] = __uint_as_float(r[0][c]);
                    }
                }
                umma::fence_before_sync();
                __syncwarp();
                const bool ring_done = C::F8 && (kk == SC_BLK - 1 || k == periods - 1);
                if (lane == 0) {
                    mbar_arrive(&acc_empty[ab]);
                    if (ring_done) mbar_arrive(&sc_empty[cs]);
                }
                if (++ab == C::NBUF) {
                    ab = 0;
                    aph ^= 1;
                }
                if (ring_done && ++cs == SC_RING) {
                    cs = 0;
                    cph ^= 1;
                }
            }
            if (ranks > 1) {
                // this CTA's part of the tile, [a][column][weight row]; NaN if a wait
                // ran out, so that the cluster's sum does not pass for a result
#pragma unroll
                for (int a = 0; a < C::NA; ++a)
#pragma unroll
                    for (int c = 0; c < C::CH; ++c)
                        if (col + c < w.nv)
                            part[(a * C::NT + col + c) * TILE_W + quad * 32 + lane] =
                                ok ? acc[a][c] : __int_as_float(0x7FC00000);
                break;
            }
            if (!ok) break;
            const int nr = w.nbi * TILE_W + quad * 32 + lane;  // this thread's weight row
            if constexpr (C::GU) {
                // a = silu(g) u; a tile's 128 rows are one scale block of the
                // activations, so the maximum over lanes and warps is the block's
                uint32_t* am = amax + par * 4 * C::NT;
                if (col < w.np) {
                    uint32_t mine = 0;
#pragma unroll
                    for (int c = 0; c < C::CH; ++c) {
                        acc[0][c] = swiglu(acc[0][c], acc[C::NA - 1][c]);
                        const uint32_t m =
                            __reduce_max_sync(0xffffffffu, finite_abs_bits(acc[0][c]));
                        if (lane == c) mine = m;
                    }
                    if (lane < C::CH) am[quad * C::NT + col + lane] = mine;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&am_full[half]);
                ok = mbar_wait_spin(&am_full[half], par, p.err, DEV_GMM_TIMEOUT);
                if (!ok) break;
                if (col < w.np) {
                    float s = 1.f, inv = 1.f;
                    if (lane < C::CH) {
                        const int j = col + lane;
                        const uint32_t m = max(max(am[j], am[C::NT + j]),
                                               max(am[2 * C::NT + j], am[3 * C::NT + j]));
                        f8_scale(m, &s, &inv);
                        if (quad == 0 && j < w.nv)
                            p.as[static_cast<int64_t>(w.row0 + j) * p.nb + w.nbi] = s;
                    }
#pragma unroll
                    for (int c = 0; c < C::CH; c += 2) {
                        const float i0 = __shfl_sync(0xffffffffu, inv, c);
                        const float i1 = __shfl_sync(0xffffffffu, inv, c + 1);
                        const uint32_t q = f8_pack2(acc[0][c] * i0, acc[0][c + 1] * i1);
                        uint8_t* dst =
                            p.aq + static_cast<int64_t>(w.row0 + col + c) * p.N + nr;
                        if (col + c < w.nv) dst[0] = static_cast<uint8_t>(q & 0xFF);
                        if (col + c + 1 < w.nv) dst[p.N] = static_cast<uint8_t>(q >> 8);
                    }
                }
            } else if (nr < p.N) {
#pragma unroll
                for (int c = 0; c < C::CH; ++c)
                    if (col + c < w.nv)
                        store_out(p.y, static_cast<int64_t>(w.row0 + col + c) * p.ldy + nr, p.out,
                                  acc[0][c]);
            }
        }
    }

    __syncwarp();
    if (ranks > 1) {
        // add the ranks' parts in rank order; rank r takes columns r, r + ranks, ...,
        // a thread one weight row
        cluster_sync();
        if (warp >= 4 && first < tiles) {
            const Tile w = w0;
            const int half = (warp - 4) >> 2, r = (tid - 128) & 127;
            const int nr = w.nbi * TILE_W + r;
            for (int j0 = 0; j0 < w.nv; j0 += 2 * ranks) {
                const int j = j0 + rank + ranks * half;
                float v[C::NA];
                if (j < w.nv) {
#pragma unroll
                    for (int a = 0; a < C::NA; ++a)
                        v[a] = cluster_sum(part + (a * C::NT + j) * TILE_W + r, ranks);
                }
                if constexpr (C::GU) {
                    float a = 0.f;
                    if (j < w.nv) a = swiglu(v[0], v[C::NA - 1]);
                    const uint32_t m = __reduce_max_sync(0xffffffffu, finite_abs_bits(a));
                    uint32_t* am = amax + ((j0 / (2 * ranks)) & 1) * 8 + half * 4;
                    if (lane == 0) am[warp & 3] = m;
                    named_bar(1 + half, 128);
                    float s, inv;
                    f8_scale(max(max(am[0], am[1]), max(am[2], am[3])), &s, &inv);
                    if (j < w.nv) {
                        p.aq[static_cast<int64_t>(w.row0 + j) * p.N + nr] =
                            static_cast<uint8_t>(f8_pack2(a * inv, 0.f) & 0xFF);
                        if (r == 0) p.as[static_cast<int64_t>(w.row0 + j) * p.nb + w.nbi] = s;
                    }
                } else if (j < w.nv && nr < p.N) {
                    store_out(p.y, static_cast<int64_t>(w.row0 + j) * p.ldy + nr, p.out, v[0]);
                }
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another may read its part
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 1) umma::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace gmm
}  // namespace qmoe
