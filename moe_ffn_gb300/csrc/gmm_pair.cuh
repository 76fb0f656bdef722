// gmm_pair.cuh — the grouped products' kernel for many rows: a pair of CTAs
// (a cluster of two) computes 256 weight rows x up to 192 token rows with
// tcgen05.mma cta_group::2.
//
// Why pairs: each CTA loads its own 128 weight rows and half of the token
// rows, so a stage of 128 bytes of K brings 32 KB per CTA for
// 128 x 256 x 128 multiply-adds.  One CTA alone would load 48 KB for the same
// work, and was bound by the 64 bytes an SM takes from L2 per clock.
//
// Scales (e4m3).  The weight rows lie along TMEM lanes and the token rows
// along its columns, so every column of a partial product has its own scale.
// The epilogue reads TMEM in 16x256b fragments, in which a thread has two of
// every eight columns of four rows: a quarter of the scale loads that
// whole-row fragments need (those took 1024 clocks of shared-memory bandwidth
// per k-block of 512 clocks).
//
// Roles (512 threads): warp 0 loads, warp 1 (of the first CTA) issues the
// MMAs, warps 2-3 copy scales, warps 4-15 are the epilogue: warp w reads
// lanes 32 (w % 4) .. + 31 and every third run of 32 columns.  A warp hands a
// TMEM buffer back once its values are in registers, before it adds them.
#pragma once
#include "gmm.cuh"

namespace qmoe {
namespace gmm {

constexpr int P_CG = 3;            // runs of columns in flight, one per four warps
constexpr int P_EPI = 4 * P_CG;    // epilogue warps
constexpr int P_THREADS = 128 + 32 * P_EPI;
constexpr int P_CH = 32;           // columns per run
// registers per thread: 128 x 56 + 384 x 152 = 65,536, the launch's 512 x 128
constexpr int P_REGS_LOAD = 56, P_REGS_EPI = 152;

template <bool F8_, int NT_, int NST_, bool GU_>
struct PairCfg {
    static constexpr bool F8 = F8_, GU = GU_;
    static constexpr int NT = NT_, NST = NST_;
    static constexpr int NA = GU ? 2 : 1;
    static constexpr int BOX = GU ? 16 : 32;  // token rows per TMA box; divides NT / 2
    static constexpr int A_BYTES = TILE_W * KBLK;
    static constexpr int STAGE = NA * A_BYTES + NT / 2 * KBLK;
    static constexpr int PARTS = NA * NT / P_CH / P_CG;  // runs per epilogue warp
    static constexpr int TM_BUF = NA * NT;
    static constexpr int TM_COLS = 512;
    static constexpr int SC_ROW = NT + 4;  // scales of x, then of W (gate, up)
    static constexpr int SC_STAGE = SC_BLK * SC_ROW;  // floats
    static constexpr int OUT_BYTES = GU ? 1024 : 2048;  // staging per epilogue warp
    static constexpr int O_SC = NST * STAGE;
    static constexpr int O_OUT = O_SC + (F8 ? SC_RING * SC_STAGE * 4 : 0);
    static constexpr int O_AMAX = O_OUT + P_EPI * OUT_BYTES;
    static constexpr int O_BAR = O_AMAX + (GU ? 2 * 4 * NT * 4 : 0);
    static constexpr int N_BAR = 2 * NST + 2 * SC_RING + 4 + 1;
    static constexpr int O_TAB = O_BAR + (N_BAR + 1) * 8;
    static constexpr int smem(int E) { return 1024 + O_TAB + (3 * E + 4) * 4; }
    static_assert(PARTS == 2 && 2 * TM_BUF <= TM_COLS && STAGE % 1024 == 0, "tile shape");
    static_assert((NT / 2) % BOX == 0, "boxes fill a stage exactly");
};

template <class C>
__global__ void __launch_bounds__(P_THREADS, 1) __cluster_dims__(2, 1, 1)
    gmm_pair_kernel(const Params p, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_w2,
                    const __grid_constant__ CUtensorMap tm_x) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* ring = reinterpret_cast<float*>(base + C::O_SC);
    uint32_t* amax = reinterpret_cast<uint32_t*>(base + C::O_AMAX);
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::O_BAR);
    uint64_t* full = bars;                    // [NST] first CTA's: both CTAs' copies landed
    uint64_t* empty = full + C::NST;          // [NST] each CTA's
    uint64_t* sc_full = empty + C::NST;
    uint64_t* sc_empty = sc_full + SC_RING;
    uint64_t* acc_full = sc_empty + SC_RING;  // [2] each CTA's
    uint64_t* acc_empty = acc_full + 2;       // [2] first CTA's: both epilogues are done
    uint64_t* mma_done = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BAR);
    int* t_lo = reinterpret_cast<int*>(base + C::O_TAB);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    if (warp == 1) umma::tmem_alloc_pair(tmem_slot, C::TM_COLS);
    if (tid == 0) {
        for (int i = 0; i < C::NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < SC_RING; ++i) {
            mbar_init(&sc_full[i], 64);
            mbar_init(&sc_empty[i], P_EPI);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * P_EPI);
        }
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    const int nbt = (p.nb + 1) / 2;  // tiles of 256 weight rows
    if (warp == 0) build_tables(p, C::NT, nbt, lane, t_lo, t_hi, t_pre);
    umma::fence_before_sync();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either is signalled
    umma::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = t_pre[p.E];
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < 4) {
        regs_dec<P_REGS_LOAD>();
        if (warp == 0) {
            // ------------------------------------------------------ loads
            int it = 0, s = 0;
            uint32_t ph = 1;  // parity of the wait for a free stage
            bool ok = true;
            const uint32_t full0 = cluster_addr(full, 0);
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const int half = w.np >> 1;
                const int boxes = (half + C::BOX - 1) / C::BOX;
                const uint32_t bytes = 2 * (C::NA * C::A_BYTES + boxes * C::BOX * KBLK);
                const int wrow = (2 * w.nbi + static_cast<int>(rank)) * TILE_W;
                const int xrow = w.row0 + static_cast<int>(rank) * half;
                for (int kb = 0; kb < p.kb; ++kb, ++it) {
                    // (before any use of a stage the wait passes at once)
                    if (!mbar_wait_spin(&empty[s], ph, p.err, DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t* st = base + s * C::STAGE;
                        const uint32_t bar = full0 + s * 8;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        const int kx = C::F8 ? kb * KBLK : kb * (KBLK / 2);
                        tma_load_3d_pair(st, &tm_w, kx, wrow, w.e, bar);
                        if constexpr (C::GU)
                            tma_load_3d_pair(st + C::A_BYTES, &tm_w2, kx, wrow, w.e, bar);
                        uint8_t* sb = st + C::NA * C::A_BYTES;
#pragma unroll
                        for (int b = 0; b < C::NT / 2 / C::BOX; ++b)
                            if (b < boxes)
                                tma_load_2d_pair(sb + b * C::BOX * KBLK, &tm_x, kx,
                                                 xrow + b * C::BOX, bar);
                    }
                    __syncwarp();
                    if (++s == C::NST) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // never leave with copies in flight (the pair's: the other CTA
            // leaves only after the cluster barrier at the end)
            if (rank == 0)
                for (int k = max(it - C::NST, 0); k < it; ++k)
                    mbar_wait_spin(&full[k % C::NST], (k / C::NST) & 1, p.err, DEV_GMM_TIMEOUT);
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------- MMA
            int s = 0;
            uint32_t ph = 0, ab = 0, aph = 1;  // stage and accumulator phases
            bool ok = true;
            const uint64_t da0 = umma::desc_sw128(smem_u32(base));
            const uint64_t db0 = umma::desc_sw128(smem_u32(base) + C::NA * C::A_BYTES);
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const uint32_t idesc = p.idesc | (static_cast<uint32_t>(w.np >> 3) << 17);
                for (int kb = 0; kb < p.kb; ++kb) {
                    const bool fresh = C::F8 || kb == 0;
                    if (fresh && !mbar_wait_spin(&acc_empty[ab], aph, p.err, DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait_spin(&full[s], ph, p.err, DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    umma::fence_after_sync();
                    const bool last = C::F8 || kb == p.kb - 1;
                    if (elect_one()) {
                        // 32 bytes of K further: the descriptors' address field + 2
                        const uint64_t da = da0 + s * (C::STAGE >> 4);
                        const uint64_t db = db0 + s * (C::STAGE >> 4);
                        const uint32_t d = tmem + ab * C::TM_BUF;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int a = 0; a < C::NA; ++a) {
                                const uint32_t acc = (!fresh || j > 0) ? 1u : 0u;
                                const uint64_t daj = da + a * (C::A_BYTES >> 4) + 2 * j;
                                if constexpr (C::F8)
                                    umma::mma_f8_pair(d + a * C::NT, daj, db + 2 * j, idesc, acc);
                                else
                                    umma::mma_f16_pair(d + a * C::NT, daj, db + 2 * j, idesc, acc);
                            }
                        umma::commit_pair(&empty[s]);
                        if (last) umma::commit_pair(&acc_full[ab]);
                    }
                    __syncwarp();
                    if (last && (ab ^= 1) == 0) aph ^= 1;
                    if (++s == C::NST) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (elect_one()) umma::commit_pair(mma_done);
            __syncwarp();
            mbar_wait_spin(mma_done, 0, p.err, DEV_GMM_TIMEOUT);
        } else if (C::F8 && warp >= 2) {
            // ----------------------------------------------------- scales
            // sx[row][kb] to ring[kb][row] by 4-byte asynchronous copies (zeros
            // past the tile's rows), with this CTA's sw[kb] behind them
            const int lt = tid - 64;
            int ch = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const int nbi = 2 * w.nbi + static_cast<int>(rank);
                const int64_t wo = (static_cast<int64_t>(w.e) * p.nb + nbi) * p.kb;
                const float* xs = p.xs + static_cast<int64_t>(w.row0) * p.kb;
                // the second half of the last weight tile may be empty
                const float* ws = (lt == 0 ? p.ws : p.ws2) + wo;
                const bool has_w = lt < C::NA && nbi < p.nb;
                for (int k0 = 0; k0 < p.kb; k0 += SC_BLK, ++ch) {
                    const int s = ch % SC_RING, round = ch / SC_RING;
                    if (round > 0 && !mbar_wait_spin(&sc_empty[s], (round - 1) & 1, p.err,
                                                     DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = smem_u32(ring + s * C::SC_STAGE);
                    const int nk = min(SC_BLK, p.kb - k0);
                    for (int j = lt; j < w.np; j += 64)
                        for (int b = 0; b < nk; ++b)
                            cp_async4(dst + (b * C::SC_ROW + j) * 4,
                                      xs + (j < w.nv ? j : 0) * static_cast<int64_t>(p.kb) + k0 + b,
                                      j < w.nv);
                    if (has_w)
                        for (int b = 0; b < nk; ++b)
                            cp_async4(dst + (b * C::SC_ROW + C::NT + lt) * 4, ws + k0 + b, true);
                    cp_async_arrive(&sc_full[s]);
                }
            }
            cp_async_drain();
        }
    } else {
        // ------------------------------------------------------- epilogue
        regs_inc<P_REGS_EPI>();
        const int quad = warp & 3, cg = (warp - 4) >> 2;
        const int lr = lane >> 2, lc = 2 * (lane & 3);  // fragment row and column
        const uint32_t tm_lane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const uint32_t acc_empty0 = cluster_addr(acc_empty, 0);
        uint8_t* stage = base + C::O_OUT + (warp - 4) * C::OUT_BYTES;
        int ab = 0, ch = 0, par = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step, par ^= 1) {
            const Tile w = tile_at(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
            const int nbi = 2 * w.nbi + static_cast<int>(rank);
            // acc[part][row half][4 i + 2 j + b]: weight row 16 half + 8 j + lr of this
            // warp's 32, column 8 i + lc + b of its run.  Parts: runs cg and
            // cg + P_CG of the columns, or run cg of gate and of up.
            float acc[2][2][16];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[q][c >> 4][c & 15] = 0.f;
            const int parts = C::GU ? (cg * P_CH < w.np ? 2 : 0)
                                    : (cg * P_CH < w.np) + ((cg + P_CG) * P_CH < w.np);
            const int periods = C::F8 ? p.kb : 1;
            for (int k = 0; k < periods; ++k, ++ab) {
                const float* sc = nullptr;
                const int kk = k % SC_BLK;
                if constexpr (C::F8) {
                    const int s = ch % SC_RING;
                    if (kk == 0 && !mbar_wait_spin(&sc_full[s], (ch / SC_RING) & 1, p.err,
                                                   DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    sc = ring + s * C::SC_STAGE + kk * C::SC_ROW;
                }
                if (!mbar_wait_spin(&acc_full[ab & 1], (ab >> 1) & 1, p.err, DEV_GMM_TIMEOUT)) {
                    ok = false;
                    break;
                }
                umma::fence_after_sync();
                const uint32_t src0 = tm_lane + (ab & 1) * C::TM_BUF + cg * P_CH;
                if (parts == 0 && lane == 0) mbar_arrive_cluster(acc_empty0 + (ab & 1) * 8);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (q < parts) {
                        uint32_t r0[16], r1[16];
                        umma::ld_16x256b_x4(src0 + q * (P_CG * P_CH), r0);
                        umma::ld_16x256b_x4(src0 + q * (P_CG * P_CH) + (16u << 16), r1);
                        float2 s[4];
                        if constexpr (C::F8) {
                            const float sw = sc[C::NT + (C::GU ? q : 0)];
                            const float* sx = sc + (C::GU ? cg : cg + P_CG * q) * P_CH + lc;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                s[i] = *reinterpret_cast<const float2*>(sx + 8 * i);
                                s[i].x *= sw;
                                s[i].y *= sw;
                            }
                        }
                        umma::wait_ld(r0);
                        umma::wait_ld(r1);
                        if (q == parts - 1) {
                            umma::fence_before_sync();
                            if (lane == 0) mbar_arrive_cluster(acc_empty0 + (ab & 1) * 8);
                        }
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            if constexpr (C::F8) {
                                fma2(acc[q][0][c], acc[q][0][c + 1], __uint_as_float(r0[c]),
                                     __uint_as_float(r0[c + 1]), s[c / 4].x, s[c / 4].y);
                                fma2(acc[q][1][c], acc[q][1][c + 1], __uint_as_float(r1[c]),
                                     __uint_as_float(r1[c + 1]), s[c / 4].x, s[c / 4].y);
                            } else {
                                acc[q][0][c] = __uint_as_float(r0[c]);
                                acc[q][0][c + 1] = __uint_as_float(r0[c + 1]);
                                acc[q][1][c] = __uint_as_float(r1[c]);
                                acc[q][1][c + 1] = __uint_as_float(r1[c + 1]);
                            }
                        }
                    }
                if constexpr (C::F8) {
                    if (kk == SC_BLK - 1 || k == periods - 1) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sc_empty[ch % SC_RING]);
                        ++ch;
                    }
                }
            }
            if (!ok) break;
            const int n0 = nbi * TILE_W + quad * 32;  // first of this warp's weight rows
            if constexpr (C::GU) {
                // a = silu(g) u; this CTA's 128 rows are one scale block of the
                // activations: maxima over a thread's rows, the lanes, the four warps
                uint32_t* am = amax + par * 4 * C::NT;
                const int col = cg * P_CH;
                if (parts > 0) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t m = 0;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int x = 4 * q + 2 * j + b;
                                    const float g = acc[0][h][x], u = acc[1][h][x];
                                    const float v = __fdividef(g, 1.0f + __expf(-g)) * u;
                                    acc[0][h][x] = v;
                                    m = max(m, finite_abs_bits(v));
                                }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                            if (lr == 0) am[quad * C::NT + col + 8 * q + lc + b] = m;
                        }
                }
                named_bar(1 + cg, 128);
                if (parts > 0) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float inv[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int j = col + 8 * q + lc + b;
                            const uint32_t m = max(max(am[j], am[C::NT + j]),
                                                   max(am[2 * C::NT + j], am[3 * C::NT + j]));
                            float s;
                            f8_scale(m, &s, &inv[b]);
                            if (quad == 0 && lr == 0 && j < w.nv && nbi < p.nb)
                                p.as[static_cast<int64_t>(w.row0 + j) * p.nb + nbi] = s;
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int x = 4 * q + 2 * j;
                                const uint32_t c = f8_pack2(acc[0][h][x] * inv[0],
                                                            acc[0][h][x + 1] * inv[1]);
                                uint8_t* d = stage + (8 * q + lc) * 32 + 16 * h + 8 * j + lr;
                                d[0] = static_cast<uint8_t>(c & 0xFF);
                                d[32] = static_cast<uint8_t>(c >> 8);
                            }
                    }
                    __syncwarp();
                    // lane = token: 32 bytes of one row of the activations
                    if (col + lane < w.nv && nbi < p.nb) {
                        const uint4* src = reinterpret_cast<const uint4*>(stage + lane * 32);
                        uint4* dst = reinterpret_cast<uint4*>(
                            p.aq + static_cast<int64_t>(w.row0 + col + lane) * p.N + n0);
                        dst[0] = src[0];
                        dst[1] = src[1];
                    }
                    __syncwarp();
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int col = (P_CG * i + cg) * P_CH;
                    if (i >= parts) continue;
                    if (p.vec_out && n0 + 32 <= p.N) {
                        // 16-bit y: transposed through shared memory, then 64-byte
                        // runs of y's rows.  Token c's four 16-byte units lie at
                        // c * 64 in an order that keeps stores and loads apart in
                        // the banks.
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const float lo = acc[i][m >> 1][4 * q + 2 * (m & 1)];
                                const float hi = acc[i][m >> 1][4 * q + 2 * (m & 1) + 1];
                                v[m] = p.out == OUT_BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
                            }
                            const int tok = 8 * q + (lane & 7), unit = lane >> 3;
                            stmatrix_x4_trans(stage + tok * 64 + ((unit ^ ((tok >> 1) & 3)) << 4),
                                              v[0], v[1], v[2], v[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int tok = 8 * q + (lane >> 2), unit = lane & 3;
                            const uint4 v = *reinterpret_cast<const uint4*>(
                                stage + tok * 64 + ((unit ^ ((tok >> 1) & 3)) << 4));
                            if (col + tok < w.nv)
                                *reinterpret_cast<uint4*>(
                                    static_cast<uint16_t*>(p.y) +
                                    static_cast<int64_t>(w.row0 + col + tok) * p.ldy + n0 +
                                    8 * unit) = v;
                        }
                        __syncwarp();
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                const int c = col + 8 * (x >> 2) + lc + (x & 1);
                                const int n = n0 + 16 * h + 8 * ((x >> 1) & 1) + lr;
                                if (c < w.nv && n < p.N)
                                    store_out(p.y, static_cast<int64_t>(w.row0 + c) * p.ldy + n,
                                              p.out, acc[i][h][x]);
                            }
                    }
                }
            }
        }
    }

    __syncwarp();
    umma::fence_before_sync();
    __syncthreads();
    // neither CTA leaves while the other may still signal it or read its copies
    cluster_sync();
    umma::fence_after_sync();
    if (warp == 1) umma::tmem_dealloc_pair(tmem, C::TM_COLS);
}

}  // namespace gmm
}  // namespace qmoe
