// w4_many.cuh — the 4-bit products' kernel for many rows per group, on the
// 5th-generation tensor cores.
//
// A tile is 256 weight rows (two halves, an MMA of 128 rows each) by up to 64 token
// rows, K in blocks of 128 columns.  The codes come by TMA.  Sixteen warps, a weight row
// to each thread, turn them into exact 16-bit integers and write them to tensor memory,
// from where the MMA takes its A operand (through shared memory every tile would be
// written and read once more): eight of them the even k-blocks, eight the odd ones.
// Token rows come by TMA too, or, where their rows are not aligned or are f32 (cut into
// three bf16 parts: three MMAs on one A), from four warps more.  The sums over the
// columns of one scale go to an accumulator of their own, which eight warps, a weight row
// to each thread again, multiply by the row's scale and add up in registers.  Where tiles
// are few the CTAs of a cluster share K and add their parts in rank order through
// distributed shared memory.
//
// Bound by the steps between the roles and by instruction issue (67%), not by the tensor
// cores (19% busy) or HBM: a k-block takes about 1,100 clocks of handing over with no
// work in it, 1,450 with.  Measured: 64 groups of 64 rows, 1024 x 2048, 37.5 us (460
// TFLOP/s, 1.9 TB/s), of 16 rows 32.8; 4096 rows in 64 uneven groups 50 us (370 tiles on
// 152 SMs are three rounds, the last of them 43% full); 14336 x 4096, 64 rows 27.8 us, 4096
// rows 665 us (723 TFLOP/s: every weight is decoded again for each 64 rows; f32 rows 2.2 ms).
// Without the products of one part (timing only, 38.3 us whole): MMAs 37.8, sums 30.3,
// codes 35.4, all three 26.4, the copies too 22.7.
#pragma once
#include "w4.cuh"

namespace qmoe {
namespace w4 {

constexpr int MANY_ROWS = 256;
constexpr int MANY_NT = 64;
constexpr unsigned NAP_NS = 200;
constexpr unsigned TRY_NS = 3760;  // a nap and a try of a barrier that does not complete

// TMA_X: token rows by TMA.
template <class X_, int S_, bool TMA_X_>
struct Many {
    using X = X_;
    static constexpr bool F32X = std::is_same<X, float>::value, TMA_X = TMA_X_;
    using H = typename std::conditional<std::is_same<X, __half>::value, __half,
                                        __nv_bfloat16>::type;
    static constexpr int S = S_, PARTS = F32X ? 3 : 1;
    static constexpr int GPB = 128 / S;            // scales of a k-block
    static constexpr int CB = 4 / GPB;             // k-blocks of a chunk of four scales
    static constexpr int XS = F32X ? 2 : 4;        // stages of token rows, a k-block each
    static constexpr int WS = 3;                   // stages of codes, two k-blocks each
    static constexpr int SR = 3;                   // stages of scales, a chunk each
    static constexpr int AB = 2, DB = 2;           // buffers in tensor memory, per half
    static constexpr int W_BYTES = MANY_ROWS * 128;
    static constexpr int X_TILE = MANY_NT * 128;   // 64 columns of a part
    static constexpr int X_BYTES = PARTS * 2 * X_TILE;
    // warps: 0-1 MMA, one to a half, 2 TMA, 3 scales if 4-7 load token rows, else 4-7
    // scales, 16 codes, 8 sums
    static constexpr int FIRST = 8;
    static constexpr int THREADS = (FIRST + 24) * 32;
    // registers per thread after the split: no more in all than the launch was given,
    // 64 for each
    static constexpr int REGS_AUX = 40, REGS_X = TMA_X ? REGS_AUX : 72, REGS_CODES = 48,
                         REGS_SUMS = TMA_X ? 120 : 104;
    static_assert(REGS_AUX + REGS_X + 4 * REGS_CODES + 2 * REGS_SUMS <= 64 * (FIRST + 24) / 4,
                  "register split");
    static constexpr int S_WARPS = TMA_X ? 4 : 1;  // for scales
    static constexpr int BATCH = F32X ? 4 : 8;     // eights of columns in flight per thread
    static constexpr int TM_A = DB * 2 * MANY_NT, TM_COLS = 512;
    static_assert(TM_A + AB * 2 * 64 <= TM_COLS, "tensor memory");
    static constexpr int O_W = XS * X_BYTES;
    static constexpr int O_S = O_W + WS * W_BYTES;
    static constexpr int O_Z = O_S + SR * 4 * MANY_ROWS * 4;
    static constexpr int O_BAR = O_Z + SR * 4 * MANY_ROWS * 2;
    static constexpr int N_BAR = 2 * (WS + XS + SR) + 4 * AB + 4 * DB;
    static constexpr int O_TAB = O_BAR + (N_BAR + 2) * 8;
    static constexpr int smem(int E) { return O_TAB + (3 * E + 1) * 4 + 1024; }
    // (a cluster's parts lie where the stages were)
    static_assert(O_S >= MANY_NT * MANY_ROWS * 4, "room for a tile");
};

// A word of eight codes in order, a[i] holds codes 2 i and 2 i + 1: both nibbles of byte i,
// the low one in the low half, the high one in bits 4..7 of the high half (the mode of
// prmt that repeats a byte's sign gives the zeros between them).
template <class H>
__device__ __forceinline__ void codes_in_order(uint32_t w, uint32_t bias, uint32_t* a) {
    constexpr uint32_t up = (Magic<H>::HIGH & 0xFFFF0000u) | (Magic<H>::LOW & 0xFFFFu);
    const uint32_t e = w & 0x0F0F0F0Fu, o = w & 0xF0F0F0F0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r;
        asm("prmt.b32 %0, %1, %2, %3;"
            : "=r"(r)
            : "r"(e), "r"(o), "r"(0x8480 + 0x1111 * i));
        a[i] = fma2<H>(r, up, bias);
    }
}

// Eight values of a row in order; an f32 row in three parts (split3).
template <class X>
__device__ __forceinline__ void in_order(const Raw8<X>& v,
                                         uint4 (&out)[std::is_same<X, float>::value ? 3 : 1]) {
    if constexpr (std::is_same<X, float>::value) {
        uint32_t h[3][8];
        split3(v, h);
#pragma unroll
        for (int q = 0; q < 3; ++q)
            out[q] = make_uint4(upper2(h[q][0], h[q][1]), upper2(h[q][2], h[q][3]),
                                upper2(h[q][4], h[q][5]), upper2(h[q][6], h[q][7]));
    } else {
        out[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    many_kernel(const Params p, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_x) {
    using X = typename C::X;
    using H = typename C::H;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tries;  // of a wait that runs out
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sc_s = reinterpret_cast<float*>(base + C::O_S);
    uint16_t* sc_z = reinterpret_cast<uint16_t*>(base + C::O_Z);
    float* part = reinterpret_cast<float*>(base);
    uint64_t* w_full = reinterpret_cast<uint64_t*>(base + C::O_BAR);
    uint64_t* w_empty = w_full + C::WS;
    uint64_t* x_full = w_empty + C::WS;
    uint64_t* x_empty = x_full + C::XS;
    uint64_t* s_full = x_empty + C::XS;
    uint64_t* s_empty = s_full + C::SR;
    uint64_t* a_full = s_empty + C::SR;     // [AB][half]
    uint64_t* a_empty = a_full + 2 * C::AB;
    uint64_t* d_full = a_empty + 2 * C::AB; // [DB][half]
    uint64_t* d_empty = d_full + 2 * C::DB;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(w_full + C::N_BAR);
    int* t_lo = reinterpret_cast<int*>(base + C::O_TAB);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == 0) umma::tmem_alloc(tmem_slot, C::TM_COLS);
    if (tid == 0) {
        for (int i = 0; i < C::WS; ++i) { mbar_init(&w_full[i], 1); mbar_init(&w_empty[i], 16); }
        for (int i = 0; i < C::XS; ++i) {
            mbar_init(&x_full[i], C::TMA_X ? 1 : 4);
            mbar_init(&x_empty[i], 2);
        }
        for (int i = 0; i < C::SR; ++i) { mbar_init(&s_full[i], C::S_WARPS); mbar_init(&s_empty[i], 24); }
        for (int i = 0; i < 2 * C::AB; ++i) { mbar_init(&a_full[i], 4); mbar_init(&a_empty[i], 1); }
        for (int i = 0; i < 2 * C::DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 4); }
        const unsigned long long tries = wait_limit(p.err) / TRY_NS + 1;
        s_tries = tries < 0xFFFFFFFFu ? static_cast<uint32_t>(tries) : 0xFFFFFFFFu;
        fence_barrier_init();
        prefetch_tensormap(&tm_w);
        if constexpr (C::TMA_X) prefetch_tensormap(&tm_x);
    }
    // failure-path tests: this CTA loads no codes, so that the waits for them run out
    const bool skip = __ldcg(&p.err->skip_arrive_cta) == static_cast<int>(blockIdx.x);
    pdl_wait();
    pdl_trigger();
    umma::fence_before_sync();
    gmm::build_tables(p, MANY_NT, p.nb, t_lo, t_hi, t_pre);
    umma::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int tiles = t_pre[p.E];

    // A cluster takes tiles first, first + step, ...; of more than one CTA, one tile,
    // each CTA a share of K.
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int lg = 31 - __clz(ranks);
    const int first = blockIdx.x >> lg;
    const int step = ranks > 1 ? max(tiles, 1) : gridDim.x;
    const int kb_all = (p.K + 127) / 128;
    const int kbeg = (rank * kb_all) >> lg, nkb = (((rank + 1) * kb_all) >> lg) - kbeg;
    auto tile_of = [&](int t) {
        return gmm::tile_at_warp(t, MANY_NT, 16, t_lo, t_hi, t_pre, p.E);
    };
    // whether a tile's half has weight rows (one without goes through the same steps,
    // its MMAs and sums left out)
    auto live = [&](const gmm::Tile& c, int h) { return c.nbi * MANY_ROWS + 128 * h < p.N; };
    // Waits.  A try itself suspends the warp, until the phase completes or for a time that the
    // hardware sets, so a second one is rare; what follows the first is kept short, for there
    // are many of these and the roles' loops share the instruction caches (with the
    // pipelines' usual longer form 43 us for 64 groups of 64 rows, 1024 x 2048, with this one
    // 39).  So the limit is a number of tries instead of a time: TRY_NS is what one took
    // (25,000 in 93.8 ms; a longer suspend-time hint does not change the hardware's part).
    // Reading the clock in this loop, in seven forms, cost 3 to 5% (37.7 -> 39.0 to 39.7
    // us).  A wait that runs out does so for the whole warp: what follows is warp-wide.
    auto wait = [&](uint64_t* b, uint32_t parity) {
        bool ok = mbar_try_wait(b, parity);
        if (__all_sync(0xffffffffu, ok)) return true;
#pragma unroll 1
        for (uint32_t i = s_tries; i > 0 && !ok; --i) {
            __nanosleep(NAP_NS);
            ok = mbar_try_wait(b, parity);
        }
        if (!ok) record_error(p.err, DEV_GMM_TIMEOUT);
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // scales: chunks of four per row, for `n` threads
    auto scales = [&](int th, int n) {
        const int SG = p.K / C::S;
        const int ss = p.stype == QMOE_F32 ? 4 : 2;
        const bool vec = SG % 4 == 0 && (kbeg * C::GPB) % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(p.scale) % (4 * ss) == 0 &&
                         reinterpret_cast<uintptr_t>(p.zero) % 4 == 0;
        uint32_t ch = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            for (int k = 0; k < nkb && ok; k += C::CB, ++ch) {
                const int g0 = (kbeg + k) * C::GPB;
                const uint32_t s = ch % C::SR;
                const bool whole = vec && g0 + 4 <= SG;
                for (int r0 = th; r0 < MANY_ROWS; r0 += 2 * n) {
                    uint4 raw[2];  // as they lie: four of 32 bits, or .x and .y two of 16 each
                    uint32_t zero[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = min(c.nbi * MANY_ROWS + r0 + j * n, p.N - 1);
                        const int64_t at = (static_cast<int64_t>(c.e) * p.N + r) * SG + g0;
                        zero[j] = 0x08080808u;
                        if (whole) {
                            if (ss == 4) {
                                raw[j] = __ldcg(reinterpret_cast<const uint4*>(
                                    static_cast<const float*>(p.scale) + at));
                            } else {
                                const uint2 q = __ldcg(reinterpret_cast<const uint2*>(
                                    static_cast<const uint16_t*>(p.scale) + at));
                                raw[j].x = q.x;
                                raw[j].y = q.y;
                            }
                            if (p.zero)
                                zero[j] = __ldcg(reinterpret_cast<const uint32_t*>(p.zero + at));
                        } else {
                            uint32_t v[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const bool in = g0 + g < SG;
                                v[g] = in ? load_raw(p.scale, at + g, p.stype) : 0u;
                                if (p.zero && in)
                                    zero[j] = (zero[j] & ~(0xFFu << (8 * g))) |
                                              (static_cast<uint32_t>(__ldcg(p.zero + at + g))
                                               << (8 * g));
                            }
                            raw[j] = ss == 4 ? make_uint4(v[0], v[1], v[2], v[3])
                                             : make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, 0, 0);
                        }
                    }
                    if (r0 == th) ok = wait(&s_empty[s], ((ch / C::SR) & 1) ^ 1);
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t v[4] = {ss == 4 ? raw[j].x : raw[j].x & 0xFFFFu,
                                               ss == 4 ? raw[j].y : raw[j].x >> 16,
                                               ss == 4 ? raw[j].z : raw[j].y & 0xFFFFu,
                                               ss == 4 ? raw[j].w : raw[j].y >> 16};
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const int at = (s * 4 + g) * MANY_ROWS + r0 + j * n;
                            sc_s[at] = scale_value(v[g], p.stype);
                            sc_z[at] = static_cast<uint16_t>(Magic<H>::bias(zero[j] >> (8 * g)));
                        }
                    }
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&s_full[s]);
            }
        }
    };

    if (warp < 4) {
        regs_dec<C::REGS_AUX>();
        if (warp < 2) {
            // -------------------------------------------------------- MMA
            const int h = warp;
            const uint64_t d0 = umma::desc_sw128(smem_u32(base));
            const uint32_t b_hi = static_cast<uint32_t>(d0 >> 32), b_lo = static_cast<uint32_t>(d0);
            const uint32_t fmt = std::is_same<X, __half>::value ? 0u : 1u;
            uint32_t xs = 0, xph = 0, db = 0, dph = 1, na0 = 0, na1 = 0, nx = 0;
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const gmm::Tile c = tile_of(t);
                const bool mine = live(c, h);
                const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) |
                                       (static_cast<uint32_t>(c.np >> 3) << 17) |
                                       ((128u >> 4) << 24);
#pragma unroll 1
                for (int k = 0; k < nkb; ++k) {
                    const uint32_t ab = k & 1, aph = (ab ? na1 : na0) & 1;
#pragma unroll
                    for (int g = 0; g < C::GPB; ++g) {
                        // all waits tried before any is acted on (before any use of a
                        // buffer the wait for it passes at once)
                        bool r0 = true, r1 = true, r2 = mbar_try_wait(&d_empty[db * 2 + h], dph);
                        if (g == 0) {
                            r0 = mbar_try_wait(&x_full[xs], xph);
                            r1 = mbar_try_wait(&a_full[ab * 2 + h], aph);
                        }
                        if (!__all_sync(0xffffffffu, r0 && r1 && r2)) {
                            if (g == 0) {
                                ok = wait(&x_full[xs], xph);
                                ok = ok && wait(&a_full[ab * 2 + h], aph);
                            }
                            ok = ok && wait(&d_empty[db * 2 + h], dph);
                            if (!ok) break;
                        }
                        umma::fence_after_sync();
                        if (elect_one()) {
                            const uint32_t d = tmem + (db * 2 + h) * MANY_NT;
                            const uint32_t a = tmem + C::TM_A + (ab * 2 + h) * 64;
                            const uint32_t b = b_lo + ((xs * C::X_BYTES) >> 4);
                            constexpr int KS = C::S / 16;
                            if (mine)
#pragma unroll
                                for (int q = C::PARTS - 1; q >= 0; --q)
#pragma unroll
                                    for (int s = g * KS; s < (g + 1) * KS; ++s)
                                        umma::mma_f16_ta(
                                            d, a + s * 8,
                                            b + (((2 * q + (s >> 2)) * C::X_TILE) >> 4) +
                                                2 * (s & 3),
                                            b_hi, idesc,
                                            (q < C::PARTS - 1 || s > g * KS) ? 1u : 0u);
                            umma::commit(&d_full[db * 2 + h]);
                            if (g == C::GPB - 1) {
                                umma::commit(&a_empty[ab * 2 + h]);
                                umma::commit(&x_empty[xs]);
                            }
                        }
                        __syncwarp();
                        if (++db == C::DB) {
                            db = 0;
                            dph ^= 1;
                        }
                    }
                    if (!ok) break;
                    ++nx;
                    if (++xs == C::XS) {
                        xs = 0;
                        xph ^= 1;
                    }
                    if (ab) ++na1; else ++na0;
                }
            }
            // Every arrival that the tensor core owes lands before the CTA ends (the
            // accumulators' are waited for by the warps that read them).
            if (ok) {
                for (uint32_t i = nx > C::XS ? nx - C::XS : 0; i < nx; ++i)
                    wait(&x_empty[i % C::XS], (i / C::XS) & 1);
                if (na0 > 0) wait(&a_empty[h], (na0 - 1) & 1);
                if (na1 > 0) wait(&a_empty[2 + h], (na1 - 1) & 1);
            } else if (nx > 0 || db > 0 || dph == 0) {
                // (after a wait that ran out the other half may never commit what these
                // barriers count: the last group's own commit says that all MMAs are done,
                // which takes a microsecond, the tries 3.7 ms)
                uint64_t* last = &d_full[(db > 0 ? db - 1 : C::DB - 1) * 2 + h];
                const uint32_t done = db > 0 ? dph ^ 1 : dph;
#pragma unroll 1
                for (int i = 0; i < 1000 && !mbar_try_wait(last, done); ++i) {}
            }
        } else if (warp == 2) {
            // -------------------------------------------------------- TMA
            uint32_t it = 0, wi = 0;
            bool ok = !skip;
            for (int t = first; t < tiles && ok; t += step) {
                const gmm::Tile c = tile_of(t);
                for (int k = 0; k < nkb && ok; ++k) {
                    if ((k & 1) == 0) {
                        const uint32_t s = wi % C::WS;
                        ok = wait(&w_empty[s], ((wi / C::WS) & 1) ^ 1);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&w_full[s], C::W_BYTES);
                            // (rows and columns past the matrix arrive as zeros)
                            tma_load_3d(base + C::O_W + s * C::W_BYTES, &tm_w, (kbeg + k) * 64,
                                        c.nbi * MANY_ROWS, c.e, &w_full[s]);
                        }
                        __syncwarp();
                        ++wi;
                    }
                    if constexpr (C::TMA_X) {
                        const uint32_t s = it % C::XS;
                        ok = wait(&x_empty[s], ((it / C::XS) & 1) ^ 1);
                        if (!ok) break;
                        if (elect_one()) {
                            uint8_t* dst = base + s * C::X_BYTES;
                            mbar_arrive_expect_tx(&x_full[s], C::X_BYTES);
                            // (rows past the tile belong to other tiles: their sums are
                            // not used; rows and columns past x arrive as zeros)
                            tma_load_2d(dst, &tm_x, (kbeg + k) * 128, c.row0, &x_full[s]);
                            tma_load_2d(dst + C::X_TILE, &tm_x, (kbeg + k) * 128 + 64, c.row0,
                                        &x_full[s]);
                        }
                        __syncwarp();
                        ++it;
                    }
                }
            }
            // never leave with copies in flight
            for (uint32_t i = wi > C::WS ? wi - C::WS : 0; i < wi; ++i)
                wait(&w_full[i % C::WS], (i / C::WS) & 1);
            for (uint32_t i = it > C::XS ? it - C::XS : 0; i < it; ++i)
                wait(&x_full[i % C::XS], (i / C::XS) & 1);
        } else if constexpr (!C::TMA_X) {
            scales(lane, 32);
        }
    } else if (C::TMA_X && warp < 8) {
        regs_dec<C::REGS_AUX>();
        scales(tid - 128, 128);
    } else if (!C::TMA_X && warp < 8) {
        // ----------------------------------------------------- token rows
        regs_inc<C::REGS_X>();
        const int th = tid - 128;
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            for (int k = 0; k < nkb && ok; ++k, ++it) {
                const uint32_t s = it % C::XS;
                uint8_t* dst = base + s * C::X_BYTES;
                const int k0 = (kbeg + k) * 128;
                const X* src = static_cast<const X*>(p.x) + static_cast<int64_t>(c.row0) * p.ldx + k0;
                const int items = c.nv * 16;  // (token, eight columns)
                for (int i0 = th; i0 < MANY_NT * 16; i0 += 128 * C::BATCH) {
                    Raw8<X> v[C::BATCH];
#pragma unroll
                    for (int b = 0; b < C::BATCH; ++b) {
                        const int i = i0 + 128 * b, o = i & 15;
                        v[b].zero();
                        if (i >= items || k0 + o * 8 >= p.K) continue;
                        const X* at = src + (i >> 4) * p.ldx + o * 8;
                        if (p.vec_x) v[b].load(at);
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const X one = ldcg_value(at + e);
                                if constexpr (C::F32X) v[b].w[e] = __float_as_uint(one);
                                else reinterpret_cast<X*>(v[b].w)[e] = one;
                            }
                    }
                    if (i0 == th) ok = wait(&x_empty[s], ((it / C::XS) & 1) ^ 1);
                    if (!ok) break;
#pragma unroll
                    for (int b = 0; b < C::BATCH; ++b) {
                        const int i = i0 + 128 * b, o = i & 15;
                        if (i >= items) continue;
                        uint4 out[C::PARTS];
                        in_order<X>(v[b], out);
                        uint8_t* at = dst + (o >> 3) * C::X_TILE +
                                      umma::sw128_offset(i >> 4, (o & 7) * 16);
#pragma unroll
                        for (int q = 0; q < C::PARTS; ++q)
                            *reinterpret_cast<uint4*>(at + q * 2 * C::X_TILE) = out[q];
                    }
                }
                if (!ok) break;
                umma::fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x_full[s]);
            }
        }
    } else if (warp < C::FIRST + 16) {
        // ---------------------------------------------------------- codes
        regs_dec<C::REGS_CODES>();
        const int set = (warp - C::FIRST) >> 3, h = ((warp - C::FIRST) >> 2) & 1;
        const int row = h * 128 + (warp & 3) * 32 + lane;
        const uint32_t a = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::TM_A +
                           (set * 2 + h) * 64;
        uint32_t wi = 0, ch = 0, na = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            const bool mine = live(c, h);
            for (int k = 0; k < nkb; ++k) {
                const int kk = k % C::CB;
                const uint32_t sr = ch % C::SR, ws = wi % C::WS;
                // (every stage is waited for in turn, by a set that has nothing in it too:
                // a wait must not be two phases ahead of its barrier)
                if (kk == 0) ok = wait(&s_full[sr], (ch / C::SR) & 1);
                if ((k & 1) == 0) ok = ok && wait(&w_full[ws], (wi / C::WS) & 1);
                if (!ok) break;
                if ((k & 1) == set) {
                    const uint8_t* wr = base + C::O_W + ws * C::W_BYTES + row * 128;
                    uint32_t bias[C::GPB];
#pragma unroll
                    for (int g = 0; g < C::GPB; ++g)
                        bias[g] = __byte_perm(
                            sc_z[(sr * 4 + kk * C::GPB + g) * MANY_ROWS + row], 0u, 0x1010);
                    ok = wait(&a_empty[set * 2 + h], (na & 1) ^ 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    if (mine)
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t r[16];
                            uint32_t b = bias[0];
#pragma unroll
                            for (int g = 1; g < C::GPB; ++g)
                                if (q * 32 / C::S == g) b = bias[g];
                            const uint4 v = *reinterpret_cast<const uint4*>(
                                wr + (((set * 4 + q) ^ (row & 7)) << 4));
                            codes_in_order<H>(v.x, b, r);
                            codes_in_order<H>(v.y, b, r + 4);
                            codes_in_order<H>(v.z, b, r + 8);
                            codes_in_order<H>(v.w, b, r + 12);
                            umma::st_32x32b_x16(a + 16 * q, r);
                        }
                    umma::wait_st();
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&a_full[set * 2 + h]);
                    ++na;
                }
                __syncwarp();
                // (a stage holds an even k-block and the odd one behind it)
                const bool pair_end = (k & 1) || k == nkb - 1;
                const bool chunk_end = kk == C::CB - 1 || k == nkb - 1;
                if (lane == 0) {
                    if (pair_end) mbar_arrive(&w_empty[ws]);
                    if (chunk_end) mbar_arrive(&s_empty[sr]);
                }
                wi += pair_end;
                ch += chunk_end;
            }
        }
    } else {
        // ----------------------------------------------------------- sums
        regs_inc<C::REGS_SUMS>();
        const int h = (warp - C::FIRST - 16) >> 2, row = h * 128 + (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t gi = 0, ch = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            const bool mine = live(c, h);
            float acc[MANY_NT];
#pragma unroll
            for (int i = 0; i < MANY_NT; ++i) acc[i] = 0.f;
            for (int k = 0; k < nkb && ok; ++k) {
                const int kk = k % C::CB;
                const uint32_t sr = ch % C::SR;
                if (kk == 0) ok = wait(&s_full[sr], (ch / C::SR) & 1);
#pragma unroll
                for (int g = 0; g < C::GPB; ++g, ++gi) {
                    const uint32_t db = gi % C::DB;
                    ok = ok && wait(&d_full[db * 2 + h], (gi / C::DB) & 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    const float s = sc_s[(sr * 4 + kk * C::GPB + g) * MANY_ROWS + row];
                    const uint32_t d = lanes + (db * 2 + h) * MANY_NT;
                    if (mine)
#pragma unroll
                        for (int q = 0; q < MANY_NT / 32; ++q)
                            if (32 * q < c.np) {
                                uint32_t r[2][16];
                                umma::ld_32x32b_x16(d + 32 * q, r[0]);
                                if (32 * q + 16 < c.np) umma::ld_32x32b_x16(d + 32 * q + 16, r[1]);
                                umma::wait_ld(r[0]);
#pragma unroll
                                for (int i = 0; i < 16; i += 2)
                                    gmm::fma2(acc[32 * q + i], acc[32 * q + i + 1], r[0][i],
                                              r[0][i + 1], s, s);
                                if (32 * q + 16 < c.np) {
                                    umma::wait_ld(r[1]);
#pragma unroll
                                    for (int i = 0; i < 16; i += 2)
                                        gmm::fma2(acc[32 * q + 16 + i], acc[32 * q + 17 + i],
                                                  r[1][i], r[1][i + 1], s, s);
                                }
                            }
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[db * 2 + h]);
                }
                __syncwarp();
                if (kk == C::CB - 1 || k == nkb - 1) {
                    if (lane == 0) mbar_arrive(&s_empty[sr]);
                    ++ch;
                }
            }
            if (ranks > 1) {
                // this CTA's part of the tile, [column][weight row], where the stages
                // were (both halves' MMAs have read them); NaN if a wait ran out, so
                // that the cluster's sum does not pass for a result
                named_bar(1, 256);
#pragma unroll
                for (int i = 0; i < MANY_NT; ++i)
                    if (i < c.nv)
                        part[i * MANY_ROWS + row] =
                            ok ? acc[i] * Magic<H>::UP : __int_as_float(0x7FC00000);
                break;
            }
            const int n = c.nbi * MANY_ROWS + row;
            if (ok && n < p.N) store_column<MANY_NT>(p, c, n, acc, Magic<H>::UP);
        }
    }

    __syncwarp();
    if (ranks > 1) {
        // the ranks' parts in rank order; rank r takes columns r, r + ranks, ...
        cluster_sync();
        if (warp >= C::FIRST + 16 && first < tiles) {
            const gmm::Tile c = tile_of(first);
            const int row = tid - (C::FIRST + 16) * 32, n = c.nbi * MANY_ROWS + row;
            // (four columns at a time: the remote loads take longer than all else)
            for (int j = rank; j < c.nv; j += 4 * ranks) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = gmm::cluster_sum(part + min(j + i * ranks, c.nv - 1) * MANY_ROWS + row,
                                            ranks);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (j + i * ranks < c.nv && n < p.N)
                        store_y(p, c.row0 + j + i * ranks, n, v[i]);
            }
        }
        __syncwarp();
        cluster_sync();  // no CTA leaves while another may read its part
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (warp == 0) umma::tmem_dealloc(tmem, C::TM_COLS);
}

}  // namespace w4
}  // namespace qmoe
