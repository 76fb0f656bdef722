// gmm_pair.cuh — the grouped products' kernel for many rows: a pair of CTAs
// (a cluster of two) computes 256 weight rows by up to 256 token rows (16-bit) or
// 192 (e4m3) with tcgen05.mma cta_group::2; SwiGLU form: 256 rows of gate and of
// up by 96.
//
// Why pairs: each CTA loads its own 128 weight rows and half of the token
// rows.  A stage of 128 bytes of K is then 32 KB per CTA for
// 128 x 256 x 64 16-bit multiply-adds; one CTA alone would load 48 KB for the
// same work, and was bound by the bytes an SM takes from L2 per clock.
//
// Scales (e4m3).  The weight rows lie along TMEM lanes and the token rows
// along its columns, so every column of a partial product has its own scale.
// The epilogue reads TMEM in 16x128b fragments, in which a thread has one of
// every four columns of four rows: a quarter of the scale loads that whole-row
// fragments need (those took 1024 clocks of shared-memory bandwidth per
// 256-column k-block of 512 clocks).  Measured over 12 warps: 32x32b 439,
// 16x128b 431, 16x256b 255 bytes per clock.
//
// No pipe bounds the e4m3 form; what is left is the epilogue's chain from one
// accumulator buffer to the next (wait, TMEM read, scales, 64 FMAs per thread,
// arrival).  2048 x 4096 x 4096, the busiest SM: 1,155 clocks per k-block of 192 columns, of
// which the tensor pipe is busy 43%, the issue slots 66%.  Shared memory could
// serve it: by the counters the MMAs read 221 wavefronts per k-block (this CTA's
// weight rows and its half of the token rows), scales and staging take 296, and
// the copies write 28 KB, 744 clocks even if they took turns.  Narrower tiles read
// the weight rows more often: four buffers of 128 columns took 760 clocks per 128.
// 256 columns do not leave the epilogue's threads the registers: 64 sums, a
// fragment of 32 values and its scales without spilling take 512 threads (any
// spill in these loops cost 15 to 30 percent).
//
// So a wide tile with few epilogue warps is for many rows per group; where
// groups fill at most 128 columns, or wide tiles leave pairs idle, four buffers
// and sixteen warps are faster (the rule and both sides' times: gmm_tiles.cuh).
//
// The 16-bit form is bound by the tensor pipe: busy 81% of a launch of 16,384 rows
// and 87% on the busiest SM of 2048 x 4096 x 4096, the fill of the pipeline and the
// last stores included.
//
// Measured: f16, 16,384 rows in 8 groups, 4096 x 4096: 327 to 345 us, 1590 to
// 1680 TFLOP/s, in short runs; 370 to 399 us in long ones, where the power limit
// lowers the clock to 1.36-1.46 GHz; e4m3, 4096 x 14336 x 4096: 301 us, 1600
// TFLOP/s, at full clock in either; 64 groups of about 64 rows, 1024 x 2048 e4m3:
// 32 us, 4.3 TB/s.
//
// Roles: warps 0 and 2 load, warp 1 (of the first CTA) issues the MMAs, warp 3
// stages scale products, the warps from 4 on are the epilogue: warp w reads
// lanes 32 (w % 4) .. + 31 and up to two runs of 32 columns (SwiGLU form: the
// same run of gate and of up).
#pragma once
#include "gmm.cuh"

namespace qmoe {
namespace gmm {

constexpr int P_CH = 32;  // columns per run

// Configuration of one instantiation.
//   F8     e4m3 operands with scales (else 16-bit)
//   NT     token tile (columns)
//   NST    pipeline stages
//   GU     two weight stacks (gate, up) and the SwiGLU + e4m3 epilogue
//   CG     runs of columns in flight, one per four epilogue warps
template <bool F8_, int NT_, int NST_, bool GU_, int CG_>
struct PairCfg {
    static constexpr bool F8 = F8_, GU = GU_;
    static constexpr int NT = NT_, NST = NST_, CG = CG_;
    static constexpr int EPI = 4 * CG;  // epilogue warps
    static constexpr int THREADS = 128 + 32 * EPI;
    // registers per thread: 128 x 80 + 384 x 144 of the launch's 512 x 128, or
    // 128 x 64 + 512 x 104 of its 640 x 96
    static constexpr int REGS_LOAD = CG == 3 ? 80 : 64, REGS_EPI = CG == 3 ? 144 : 104;
    static constexpr int NA = GU ? 2 : 1;
    static constexpr int BOX = NT % 64 ? 16 : 32;  // token rows per TMA box; divides NT / 2
    static constexpr int A_BYTES = TILE_W * KBLK;
    static constexpr int STAGE = NA * A_BYTES + NT / 2 * KBLK;
    static constexpr int TM_BUF = NA * NT;
    static constexpr int TM_COLS = 512;
    static constexpr int NBUF = TM_COLS / TM_BUF;  // accumulator buffers
    static constexpr int SC_STAGE = SC_BLK * NA * NT;  // floats: sx sw of every column
    // staging per epilogue warp: 32 tokens of 32 values
    static constexpr int OUT_BYTES = GU ? 1024 : 2048;
    static constexpr int O_SC = NST * STAGE;
    static constexpr int O_OUT = O_SC + (F8 ? SC_RING * SC_STAGE * 4 : 0);
    static constexpr int O_AMAX = O_OUT + EPI * OUT_BYTES;
    static constexpr int O_BAR = O_AMAX + (GU ? 2 * 4 * NT * 4 : 0);
    static constexpr int N_BAR = 2 * NST + 2 * SC_RING + 2 * NBUF + 1 + (GU ? CG : 0);
    static constexpr int O_TAB = O_BAR + (N_BAR + 1) * 8;
    static constexpr int smem(int E) { return 1024 + O_TAB + (3 * E + 4) * 4; }
    static_assert(TM_BUF * NBUF <= TM_COLS && STAGE % 1024 == 0, "tile shape");
    static_assert((NT / 2) % BOX == 0, "boxes fill a stage exactly");
    static_assert(!F8 || TM_BUF <= 2 * CG * P_CH, "at most two runs per warp");
    static_assert(CG == 3 || CG == 4, "register shares");
    static_assert(NT % P_CH == 0, "whole runs");
};

// Where token j's scale lies in a row of the ring: a thread's eight columns of
// a run (4 i + lane % 4) are consecutive.
__device__ __forceinline__ int sc_slot(int j) {
    return (j & ~31) | ((j & 3) << 3) | ((j >> 2) & 7);
}

// A run of 32 columns of this warp's 32 weight rows.
struct Frag {
    uint32_t lo[16], hi[16];  // row halves
};
__device__ __forceinline__ void frag_load(uint32_t src, Frag& f) {
    umma::ld_16x128b_x8(src, f.lo);
    umma::ld_16x128b_x8(src + (16u << 16), f.hi);
}
__device__ __forceinline__ void frag_wait(Frag& f) {
    umma::wait_ld(f.lo);
    umma::wait_ld(f.hi);
}

// 16-bit y of one run (v[row half][2 i + j]: row 16 half + 8 j + lane / 4,
// column 4 i + lane % 4), transposed through shared memory: a word holds rows r
// and r + 8 of a token; token c's 64 bytes lie at 64 c, the halves swapped
// where c has bit 1 (four tokens' words then fall in distinct banks).
__device__ __forceinline__ void store_run16(uint8_t* stage, const float (&v)[2][16], bool bf16,
                                            int lane, uint16_t* y, int64_t ldy, int nv) {
    const int lr = lane >> 2, lc = lane & 3;
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int tok = 4 * k + lc;
            *reinterpret_cast<uint32_t*>(stage + tok * 64 +
                                         ((32 * h + 4 * lr) ^ ((tok & 2) << 4))) =
                bf16 ? pack_bf16(v[h][2 * k], v[h][2 * k + 1])
                     : pack_f16(v[h][2 * k], v[h][2 * k + 1]);
        }
    __syncwarp();
    // two lanes per token, 16 rows each: 32-byte runs of y's rows
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int tok = 16 * k + (lane >> 1), h = lane & 1;
        const uint8_t* src = stage + tok * 64 + ((32 * h) ^ ((tok & 2) << 4));
        const uint4 a = *reinterpret_cast<const uint4*>(src);
        const uint4 b = *reinterpret_cast<const uint4*>(src + 16);
        if (tok < nv) {
            uint4* dst = reinterpret_cast<uint4*>(y + tok * ldy + 16 * h);
            dst[0] = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
            dst[1] = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
        }
    }
    __syncwarp();
}

// One run of y: nv tokens from y's element `first`, weight rows n0 .. n0 + 31.
__device__ __forceinline__ void store_run(const Params& p, uint8_t* stage, const float (&v)[2][16],
                                          int lane, int64_t row, int nv, int n0) {
    if (nv <= 0) return;
    if (p.vec_out && n0 + 32 <= p.N) {
        store_run16(stage, v, p.out == OUT_BF16, lane,
                    static_cast<uint16_t*>(p.y) + row * p.ldy + n0, p.ldy, nv);
        return;
    }
    // otherwise as f32 through shared memory, a row half at a time: runs of 16
    // values of y's rows
    float* f = reinterpret_cast<float*>(stage);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
            f[(4 * (x >> 1) + (lane & 3)) * 16 + 8 * (x & 1) + (lane >> 2)] = v[h][x];
        __syncwarp();
        const int n = n0 + 16 * h + (lane & 15);
        int64_t o = (row + (lane >> 4)) * p.ldy + n;
#pragma unroll 2
        for (int i = lane >> 4; i < nv && i < 32; i += 2, o += 2 * p.ldy)
            if (n < p.N) store_out(p.y, o, p.out, f[i * 16 + (lane & 15)]);
        __syncwarp();
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) __cluster_dims__(2, 1, 1)
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
    uint64_t* acc_full = sc_empty + SC_RING;  // [NBUF] each CTA's
    uint64_t* acc_empty = acc_full + C::NBUF; // [NBUF] first CTA's: both epilogues have read it
    uint64_t* mma_done = acc_empty + C::NBUF;
    uint64_t* am_full = mma_done + 1;  // [CG] SwiGLU form: four warps' maxima are there
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::N_BAR);
    int* t_lo = reinterpret_cast<int*>(base + C::O_TAB);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;

    __shared__ int notes[C::EPI][3];  // an epilogue warp's tile
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
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_empty[i], C::EPI);
        }
        for (int i = 0; i < C::NBUF; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * C::EPI);
        }
        mbar_init(mma_done, 1);
        if constexpr (C::GU)
            for (int i = 0; i < C::CG; ++i) mbar_init(&am_full[i], 4);
        fence_barrier_init();
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_x);
        if constexpr (C::GU) prefetch_tensormap(&tm_w2);
    }
    // (failure-path tests, as in gmm_kernel)
    const bool skip = __ldcg(&p.err->skip_arrive_cta) == static_cast<int>(blockIdx.x);
    pdl_wait();
    pdl_trigger();
    umma::fence_before_sync();
    build_tables(p, C::NT, (p.nb + 1) / 2, t_lo, t_hi, t_pre);
    cluster_sync();  // both CTAs' barriers exist before either is signalled
    umma::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = t_pre[p.E];
    const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (warp < 4) {
        regs_dec<C::REGS_LOAD>();
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------------ loads
            // warp 0 the weights, warp 2 the token rows: one warp issuing both
            // was as slow as the MMAs of a stage
            const bool wgt = warp == 0;
            int it = 0, s = 0;
            uint32_t ph = 1;  // parity of the wait for a free stage
            bool ok = !skip;
            const uint32_t full0 = cluster_addr(full, 0);
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at_warp(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const int half = w.np >> 1;
                const int boxes = (half + C::BOX - 1) / C::BOX;
                const uint32_t bytes = 2 * (C::NA * C::A_BYTES + boxes * C::BOX * KBLK);
                const int y = wgt ? (2 * w.nbi + static_cast<int>(rank)) * TILE_W
                                  : w.row0 + static_cast<int>(rank) * half;
                int kx = 0;  // coordinates along K: multiples of 128 bytes
                for (int kb = 0; kb < p.kb; ++kb, ++it) {
                    // (before any use of a stage the wait passes at once)
                    if (!mbar_wait_spin(&empty[s], ph, p.err, DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t* st = base + s * C::STAGE;
                        const uint32_t bar = full0 + s * 8;
                        if (wgt) {
                            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                            tma_load_3d_pair(st, &tm_w, kx, y, w.e, bar);
                            if constexpr (C::GU)
                                tma_load_3d_pair(st + C::A_BYTES, &tm_w2, kx, y, w.e, bar);
                        } else {
                            st += C::NA * C::A_BYTES;
#pragma unroll
                            for (int b = 0; b < C::NT / 2 / C::BOX; ++b)
                                if (b < boxes)
                                    tma_load_2d_pair(st + b * C::BOX * KBLK, &tm_x, kx,
                                                     y + b * C::BOX, bar);
                        }
                    }
                    __syncwarp();
                    kx += C::F8 ? KBLK : KBLK / 2;
                    if (++s == C::NST) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // never leave with copies in flight (the pair's: the other CTA
            // leaves only after the cluster barrier at the end)
            if (wgt && rank == 0)
                for (int k = max(it - C::NST, 0); k < it; ++k)
                    mbar_wait_spin(&full[k % C::NST], (k / C::NST) & 1, p.err, DEV_GMM_TIMEOUT);
        } else if (warp == 1 && rank == 0) {
            // -------------------------------------------------------- MMA
            int s = 0;
            uint32_t ph = 0, aph = ~0u;  // stage phase; a phase bit per accumulator buffer
            uint32_t ab = C::NBUF - 1;
            bool ok = true;
            const uint64_t da0 = umma::desc_sw128(smem_u32(base));
            const uint32_t hi = static_cast<uint32_t>(da0 >> 32), lo0 = static_cast<uint32_t>(da0);
            uint32_t lo = lo0;  // the stage's descriptor, low word
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at_warp(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const uint32_t idesc = p.idesc | (static_cast<uint32_t>(w.np >> 3) << 17);
                const int ret = p.kb - unreturned<C::NST>(
                                           static_cast<int64_t>((tiles - 1 - t) / step) * p.kb);
                if constexpr (!C::F8) ab = (ab + 1) % C::NBUF;
#pragma unroll 1
                for (int k0 = 0; k0 < p.kb && ok; k0 += C::NBUF) {
#pragma unroll
                    for (int k = 0; k < C::NBUF; ++k) {
                        if (k0 + k >= p.kb) break;
                        if constexpr (C::F8) ab = ab == C::NBUF - 1 ? 0 : ab + 1;
                        const bool fresh = C::F8 || k0 + k == 0;
                        const bool last = C::F8 || k0 + k == p.kb - 1;
                        // both waits tried before either is acted on
                        bool r0 = mbar_try_wait(&full[s], ph), r1 = true;
                        if (fresh) r1 = mbar_try_wait(&acc_empty[ab], (aph >> ab) & 1);
                        if (!r0) r0 = mbar_wait_spin(&full[s], ph, p.err, DEV_GMM_TIMEOUT);
                        if (!r1)
                            r1 = mbar_wait_spin(&acc_empty[ab], (aph >> ab) & 1, p.err,
                                                DEV_GMM_TIMEOUT);
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
                                for (int a = 0; a < C::NA; ++a) {
                                    const uint32_t acc = (!fresh || j > 0) ? 1u : 0u;
                                    const uint32_t aj = lo + a * (C::A_BYTES >> 4) + 2 * j;
                                    const uint32_t bj = lo + C::NA * (C::A_BYTES >> 4) + 2 * j;
                                    umma::mma_pair<C::F8>(d + a * C::NT, aj, bj, hi, idesc, acc);
                                }
                            if (k0 + k < ret) umma::commit_pair(&empty[s]);
                            if (last) umma::commit_pair(&acc_full[ab]);
                        }
                        __syncwarp();
                        if (last) aph ^= 1u << ab;
                        lo += C::STAGE >> 4;
                        if (++s == C::NST) {
                            s = 0;
                            ph ^= 1;
                            lo = lo0;
                        }
                    }
                }
            }
            if (elect_one()) umma::commit_pair(mma_done);
            __syncwarp();
            mbar_wait_spin(mma_done, 0, p.err, DEV_GMM_TIMEOUT);
        } else if (C::F8 && warp == 3) {
            // ----------------------------------------------------- scales
            // ring[kb][column] = sx[column][kb] sw[kb] (0 past the tile's rows),
            // four k-blocks at a time
            const bool vec = (p.kb & 3) == 0 && (reinterpret_cast<uintptr_t>(p.xs) & 15) == 0;
            int s = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const Tile w = tile_at_warp(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const int nbi = 2 * w.nbi + static_cast<int>(rank);
                const bool rows_in = nbi < p.nb;  // the last weight tile's second half may be empty
                const int64_t wo = (static_cast<int64_t>(w.e) * p.nb + nbi) * p.kb;
                const float* xs = p.xs + (static_cast<int64_t>(w.row0) + lane) * p.kb;
                float ws[C::NA];  // weight scales of 32 k-blocks, one per lane
                for (int k0 = 0; k0 < p.kb; k0 += SC_BLK) {
                    if ((k0 & 31) == 0)
#pragma unroll
                        for (int a = 0; a < C::NA; ++a)
                            ws[a] = rows_in && k0 + lane < p.kb
                                        ? __ldcg((a ? p.ws2 : p.ws) + wo + k0 + lane)
                                        : 0.f;
                    if (!mbar_wait_spin(&sc_empty[s], ph, p.err, DEV_GMM_TIMEOUT)) {
                        ok = false;
                        break;
                    }
                    float* dst = ring + s * C::SC_STAGE;
                    float v[C::NT / 32][SC_BLK];
#pragma unroll
                    for (int i = 0; i < C::NT / 32; ++i) {
                        const float* src = xs + static_cast<int64_t>(32 * i) * p.kb + k0;
                        const bool in = lane + 32 * i < w.nv;
                        if (vec && in) {
                            const float4 q = __ldcg(reinterpret_cast<const float4*>(src));
                            v[i][0] = q.x; v[i][1] = q.y; v[i][2] = q.z; v[i][3] = q.w;
                        } else {
#pragma unroll
                            for (int b = 0; b < SC_BLK; ++b)
                                v[i][b] = in && k0 + b < p.kb ? __ldcg(src + b) : 0.f;
                        }
                    }
#pragma unroll
                    for (int b = 0; b < SC_BLK; ++b)
#pragma unroll
                        for (int a = 0; a < C::NA; ++a) {
                            const float g = __shfl_sync(0xffffffffu, ws[a], (k0 & 31) + b);
#pragma unroll
                            for (int i = 0; i < C::NT / 32; ++i)
                                dst[(b * C::NA + a) * C::NT + sc_slot(lane + 32 * i)] =
                                    v[i][b] * g;
                        }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_full[s]);
                    if (++s == SC_RING) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------- epilogue
        regs_inc<C::REGS_EPI>();
        const int quad = warp & 3, cg = (warp - 4) >> 2;
        const int lr = lane >> 2, lc = lane & 3;  // fragment row and column
        const uint32_t acc_empty0 = cluster_addr(acc_empty, 0);
        // this warp's first run: its column among the tokens, its buffer column
        const int run_col = cg * P_CH;
        const uint32_t tm_run = tmem + (static_cast<uint32_t>(quad * 32) << 16) + run_col;
        // column distance of the two runs, in the buffer and in the ring
        constexpr int R2 = C::GU ? C::NT : C::CG * P_CH;
        uint8_t* stage = base + C::O_OUT + (warp - 4) * C::OUT_BYTES;
        volatile int* note = notes[warp - 4];
        uint32_t ab = C::NBUF - 1, aph = 0, cs = 0, cph = 0, par = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step, par ^= 1) {
            if constexpr (!C::F8) {
                const Tile w = tile_at_warp(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                const int n0 = (2 * w.nbi + static_cast<int>(rank)) * TILE_W + quad * 32;
                ab = (ab + 1) % C::NBUF;
                ok = mbar_wait_spin(&acc_full[ab], (aph >> ab) & 1, p.err, DEV_GMM_TIMEOUT);
                if (!ok) break;
                aph ^= 1u << ab;
                umma::fence_after_sync();
                if (run_col >= w.np && lane == 0) mbar_arrive_cluster(acc_empty0 + ab * 8);
#pragma unroll 1
                for (int col = run_col; col < w.np; col += R2) {
                    Frag f;
                    frag_load(tm_run + ab * C::TM_BUF + col - run_col, f);
                    frag_wait(f);
                    if (col + R2 >= w.np) {
                        umma::fence_before_sync();
                        if (lane == 0) mbar_arrive_cluster(acc_empty0 + ab * 8);
                    }
                    float v[2][16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        v[0][c] = __uint_as_float(f.lo[c]);
                        v[1][c] = __uint_as_float(f.hi[c]);
                    }
                    store_run(p, stage, v, lane, w.row0 + col, w.nv - col, n0);
                }
            } else {
                // acc[run][row half][2 i + j]: weight row 16 half + 8 j + lr of this warp's
                // 32, column 4 i + lc of the run
                constexpr int RUNS = C::GU || C::NT > C::CG * P_CH ? 2 : 1;
                float acc[RUNS][2][16];
#pragma unroll
                for (int c = 0; c < RUNS * 32; ++c) acc[c >> 5][(c >> 4) & 1][c & 15] = 0.f;
                // (the tile's fields wait in shared memory: they would take registers
                // through the K loop)
                int np;
                {
                    const Tile w = tile_at_warp(t, C::NT, 32, t_lo, t_hi, t_pre, p.E);
                    np = w.np;
                    if (lane == 0) {
                        note[0] = w.nbi;
                        note[1] = w.row0;
                        note[2] = w.nv;
                    }
                }
                const int runs = C::GU ? (run_col < np ? 2 : 0)
                                       : (run_col < np) + (RUNS > 1 && run_col + R2 < np);
                const float* run = ring + run_col + lc * 8;
#pragma unroll 1
                for (int k0 = 0; k0 < p.kb; k0 += SC_BLK) {
                    ok = mbar_wait_spin(&sc_full[cs], cph, p.err, DEV_GMM_TIMEOUT);
                    if (!ok) break;
                    const float* row = run + cs * C::SC_STAGE;
                    const int nk = min(SC_BLK, p.kb - k0);
#pragma unroll 1
                    for (int k = 0; k < nk; ++k, row += C::NA * C::NT) {
                        ab = ab == C::NBUF - 1 ? 0 : ab + 1;
                        ok = mbar_wait_spin(&acc_full[ab], (aph >> ab) & 1, p.err,
                                            DEV_GMM_TIMEOUT);
                        if (!ok) break;
                        aph ^= 1u << ab;
                        umma::fence_after_sync();
                        const uint32_t src = tm_run + ab * C::TM_BUF;
#pragma unroll
                        for (int q = 0; q < RUNS; ++q)
                            if (q < runs) {
                                Frag f;
                                frag_load(src + q * R2, f);
                                const float4* sx = reinterpret_cast<const float4*>(row + q * R2);
                                const float4 s0 = sx[0], s1 = sx[1];
                                const float s[8] = {s0.x, s0.y, s0.z, s0.w,
                                                    s1.x, s1.y, s1.z, s1.w};
                                frag_wait(f);
                                if (q == runs - 1) {
                                    umma::fence_before_sync();
                                    if (lane == 0) mbar_arrive_cluster(acc_empty0 + ab * 8);
                                }
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    acc[q][0][c] =
                                        fmaf(__uint_as_float(f.lo[c]), s[c / 2], acc[q][0][c]);
                                    acc[q][1][c] =
                                        fmaf(__uint_as_float(f.hi[c]), s[c / 2], acc[q][1][c]);
                                }
                            }
                        if (runs == 0 && lane == 0) mbar_arrive_cluster(acc_empty0 + ab * 8);
                    }
                    if (!ok) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sc_empty[cs]);
                    if (++cs == SC_RING) {
                        cs = 0;
                        cph ^= 1;
                    }
                }
                if (!ok) break;
                __syncwarp();
                const Tile w = {0, note[0], note[1], note[2], 0};
                const int nbi = 2 * w.nbi + static_cast<int>(rank);
                const int n0 = nbi * TILE_W + quad * 32;  // first of this warp's weight rows
                if constexpr (!C::GU) {
#pragma unroll
                    for (int q = 0; q < RUNS; ++q)
                        store_run(p, stage, acc[q], lane, w.row0 + run_col + q * R2,
                                  w.nv - run_col - q * R2, n0);
                } else {
                    // a = silu(g) u; this CTA's 128 rows are one scale block of the
                    // activations: maxima over a thread's rows, the lanes, the four warps
                    uint32_t* am = amax + par * 4 * C::NT;
                    if (runs > 0) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            uint32_t m = 0;
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float g = acc[0][r >> 1][2 * i + (r & 1)];
                                const float u = acc[RUNS - 1][r >> 1][2 * i + (r & 1)];
                                const float v = swiglu(g, u);
                                acc[0][r >> 1][2 * i + (r & 1)] = v;
                                m = max(m, finite_abs_bits(v));
                            }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                            if (lr == 0) am[quad * C::NT + run_col + 4 * i + lc] = m;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&am_full[cg]);
                    ok = mbar_wait_spin(&am_full[cg], par, p.err, DEV_GMM_TIMEOUT);
                    if (!ok) break;
                    if (runs > 0) {
                        uint32_t* codes = reinterpret_cast<uint32_t*>(stage);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int j = run_col + 4 * i + lc;
                            const uint32_t m = max(max(am[j], am[C::NT + j]),
                                                   max(am[2 * C::NT + j], am[3 * C::NT + j]));
                            float s, inv;
                            f8_scale(m, &s, &inv);
                            if (quad == 0 && lr == 0 && j < w.nv && nbi < p.nb)
                                p.as[static_cast<int64_t>(w.row0 + j) * p.nb + nbi] = s;
                            // one word: rows lr, lr + 8, lr + 16, lr + 24 of token 4 i + lc
                            codes[(4 * i + lc) * 8 + lr] =
                                f8_pack2(acc[0][0][2 * i] * inv, acc[0][0][2 * i + 1] * inv) |
                                (f8_pack2(acc[0][1][2 * i] * inv, acc[0][1][2 * i + 1] * inv)
                                 << 16);
                        }
                        __syncwarp();
                        // lane = token: its eight words' bytes in row order, 32 bytes of
                        // one row of the activations
                        if (run_col + lane < w.nv && nbi < p.nb) {
                            const uint4 a = *reinterpret_cast<const uint4*>(codes + lane * 8);
                            const uint4 b = *reinterpret_cast<const uint4*>(codes + lane * 8 + 4);
                            // bytes k, k+8, k+16, k+24 of word k -> four runs of eight
                            const uint32_t a01 = __byte_perm(a.x, a.y, 0x5140),
                                           a23 = __byte_perm(a.z, a.w, 0x5140),
                                           b01 = __byte_perm(b.x, b.y, 0x5140),
                                           b23 = __byte_perm(b.z, b.w, 0x5140),
                                           c01 = __byte_perm(a.x, a.y, 0x7362),
                                           c23 = __byte_perm(a.z, a.w, 0x7362),
                                           d01 = __byte_perm(b.x, b.y, 0x7362),
                                           d23 = __byte_perm(b.z, b.w, 0x7362);
                            uint4* dst = reinterpret_cast<uint4*>(
                                p.aq + static_cast<int64_t>(w.row0 + run_col + lane) * p.N + n0);
                            dst[0] = make_uint4(__byte_perm(a01, a23, 0x5410),
                                                __byte_perm(b01, b23, 0x5410),
                                                __byte_perm(a01, a23, 0x7632),
                                                __byte_perm(b01, b23, 0x7632));
                            dst[1] = make_uint4(__byte_perm(c01, c23, 0x5410),
                                                __byte_perm(d01, d23, 0x5410),
                                                __byte_perm(c01, c23, 0x7632),
                                                __byte_perm(d01, d23, 0x7632));
                        }
                    }
                    __syncwarp();  // the codes are read before the next tile's are written
                }
            }
        }
    }

    __syncwarp();
    umma::fence_before_sync();
    __syncthreads();
    // neither CTA leaves while the other's threads may still signal it or its copies
    // are read
    cluster_sync();
    umma::fence_after_sync();
    if (warp == 1) {
        // The last commit arrives in both CTAs; the first has seen its own copy before
        // the barrier above, so the second's is due now.  (Waited for here, for a
        // wait from the start of a long launch would run out.)
        if (rank != 0) mbar_wait_spin(mma_done, 0, p.err, DEV_GMM_TIMEOUT);
        __syncwarp();
        umma::tmem_dealloc_pair(tmem, C::TM_COLS);
    }
}

}  // namespace gmm
}  // namespace qmoe
