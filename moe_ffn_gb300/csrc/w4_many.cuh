// w4_many.cuh — the 4-bit products' kernel for many rows per group, on the
// 5th-generation tensor cores.
//
// A tile is 256 weight rows (two MMAs of 128) by up to 64 token rows, K in blocks of
// 128 columns.  The codes come by TMA; eight worker warps, a weight row to each thread,
// turn them into exact 16-bit integers (w4.cuh) and write them to tensor memory, from
// where the MMA takes its A operand: shared memory would be written and read once more.
// Token rows are staged by four warps, in the order of columns that the codes' bits
// give (and cut into three bf16 parts if they are f32: three MMAs on one A).  The sums
// over the columns of one scale go to an accumulator of their own, and the workers, one
// k-block behind, multiply them by the row's scale, one value per thread, and add them
// up in registers.  Where tiles are few the CTAs of a cluster share K and add their
// parts in rank order through distributed shared memory.
#pragma once
#include "w4.cuh"

namespace qmoe {
namespace w4 {

constexpr int MANY_THREADS = 512;
constexpr int MANY_ROWS = 256;
constexpr int MANY_NT = 64;

template <class X, int S_>
struct Many {
    static constexpr bool F32X = std::is_same<X, float>::value;
    static constexpr int S = S_, PARTS = F32X ? 3 : 1;
    static constexpr int GPB = 128 / S;            // scales of a k-block
    static constexpr int CB = 4 / GPB;             // k-blocks of a chunk of four scales
    static constexpr int XS = F32X ? 2 : 4;        // stages of token rows
    static constexpr int WS = 6;                   // stages of codes
    static constexpr int SR = 3;                   // stages of scales
    static constexpr int AB = 2, DB = 2;           // buffers in tensor memory, per half
    static constexpr int W_BYTES = MANY_ROWS * 64;
    static constexpr int X_TILE = MANY_NT * 128;   // 64 columns of a part
    static constexpr int X_BYTES = PARTS * 2 * X_TILE;
    static constexpr int BATCH = F32X ? 8 : 16;    // eights of columns in flight per thread
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

template <class C, class X>
__global__ void __launch_bounds__(MANY_THREADS, 1)
    many_kernel(const Params p, const __grid_constant__ CUtensorMap tm_w) {
    using H = typename std::conditional<std::is_same<X, __half>::value, __half,
                                        __nv_bfloat16>::type;
    extern __shared__ uint8_t smem_raw[];
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
    uint64_t* a_full = s_empty + C::SR;     // [half][AB]
    uint64_t* a_empty = a_full + 2 * C::AB;
    uint64_t* d_full = a_empty + 2 * C::AB; // [half][DB]
    uint64_t* d_empty = d_full + 2 * C::DB;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(w_full + C::N_BAR);
    int* t_lo = reinterpret_cast<int*>(base + C::O_TAB);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == 0) umma::tmem_alloc(tmem_slot, C::TM_COLS);
    if (tid == 0) {
        for (int i = 0; i < C::WS; ++i) { mbar_init(&w_full[i], 1); mbar_init(&w_empty[i], 8); }
        for (int i = 0; i < C::XS; ++i) { mbar_init(&x_full[i], 2); mbar_init(&x_empty[i], 1); }
        for (int i = 0; i < C::SR; ++i) { mbar_init(&s_full[i], 2); mbar_init(&s_empty[i], 8); }
        for (int i = 0; i < 2 * C::AB; ++i) { mbar_init(&a_full[i], 4); mbar_init(&a_empty[i], 1); }
        for (int i = 0; i < 2 * C::DB; ++i) { mbar_init(&d_full[i], 1); mbar_init(&d_empty[i], 4); }
        fence_barrier_init();
        prefetch_tensormap(&tm_w);
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
    const int kbeg = (rank * kb_all) >> lg, kend = ((rank + 1) * kb_all) >> lg;
    auto tile_of = [&](int t) {
        return gmm::tile_at_warp(t, MANY_NT, 16, t_lo, t_hi, t_pre, p.E);
    };
    // whether a tile's half has weight rows at all
    auto live = [&](const gmm::Tile& c, int h) { return c.nbi * MANY_ROWS + 128 * h < p.N; };
    auto wait = [&](uint64_t* b, uint32_t parity) {
        return mbar_wait_spin(b, parity, p.err, DEV_GMM_TIMEOUT);
    };

    if (warp == 0) {
        // ------------------------------------------------------------ MMA
        const uint64_t d0 = umma::desc_sw128(smem_u32(base));
        const uint32_t b_hi = static_cast<uint32_t>(d0 >> 32), b_lo = static_cast<uint32_t>(d0);
        const uint32_t fmt = std::is_same<X, __half>::value ? 0u : 1u;
        uint32_t na[2] = {0, 0}, nd[2] = {0, 0}, it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) |
                                   (static_cast<uint32_t>(c.np >> 3) << 17) | ((128u >> 4) << 24);
            for (int kb = kbeg; kb < kend && ok; ++kb, ++it) {
                const uint32_t xs = it % C::XS;
                ok = wait(&x_full[xs], (it / C::XS) & 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!live(c, h)) continue;
                    const uint32_t ab = na[h] % C::AB;
                    ok = ok && wait(&a_full[h * C::AB + ab], (na[h] / C::AB) & 1);
#pragma unroll
                    for (int g = 0; g < C::GPB; ++g) {
                        const uint32_t db = nd[h] % C::DB;
                        // (before any use of a buffer the wait passes at once)
                        ok = ok && wait(&d_empty[h * C::DB + db], ((nd[h] / C::DB) & 1) ^ 1);
                        if (!ok) break;
                        umma::fence_after_sync();
                        if (elect_one()) {
                            const uint32_t d = tmem + (db * 2 + h) * MANY_NT;
                            const uint32_t a = tmem + C::TM_A + (ab * 2 + h) * 64;
                            constexpr int KS = C::S / 16;
#pragma unroll
                            for (int q = C::PARTS - 1; q >= 0; --q)
#pragma unroll
                                for (int k = g * KS; k < (g + 1) * KS; ++k)
                                    umma::mma_f16_ta(
                                        d, a + k * 8,
                                        b_lo + ((xs * C::X_BYTES + (2 * q + (k >> 2)) * C::X_TILE) >> 4) +
                                            2 * (k & 3),
                                        b_hi, idesc, (q < C::PARTS - 1 || k > g * KS) ? 1u : 0u);
                            umma::commit(&d_full[h * C::DB + db]);
                            if (g == C::GPB - 1) umma::commit(&a_empty[h * C::AB + ab]);
                        }
                        __syncwarp();
                        ++nd[h];
                    }
                    ++na[h];
                }
                if (ok && elect_one()) umma::commit(&x_empty[xs]);
                __syncwarp();
            }
        }
        // Every arrival that the tensor core owes lands before the CTA ends (the
        // accumulators' are waited for by the workers).
        if (ok) {
            for (uint32_t i = it > C::XS ? it - C::XS : 0; i < it; ++i)
                wait(&x_empty[i % C::XS], (i / C::XS) & 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                for (uint32_t i = na[h] > C::AB ? na[h] - C::AB : 0; i < na[h]; ++i)
                    wait(&a_empty[h * C::AB + i % C::AB], (i / C::AB) & 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- codes
        uint32_t it = 0;
        bool ok = !skip;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            for (int kb = kbeg; kb < kend && ok; ++kb) {
                const uint32_t s = it % C::WS;
                ok = wait(&w_empty[s], ((it / C::WS) & 1) ^ 1);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&w_full[s], C::W_BYTES);
                    // (rows and columns past the matrix arrive as zeros)
                    tma_load_3d(base + C::O_W + s * C::W_BYTES, &tm_w, kb * 64, c.nbi * MANY_ROWS,
                                c.e, &w_full[s]);
                }
                __syncwarp();
                ++it;
            }
        }
        // never leave with copies in flight
        for (uint32_t i = it > C::WS ? it - C::WS : 0; i < it; ++i)
            wait(&w_full[i % C::WS], (i / C::WS) & 1);
    } else if (warp < 6) {
        // ----------------------------------------------------- token rows
        // two pairs of warps, one for even and one for odd k-blocks
        const uint32_t pair = (warp - 2) >> 1;
        const int th = (tid - 64) & 63;
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            for (int kb = kbeg; kb < kend && ok; ++kb, ++it) {
                if ((it & 1) != pair) continue;
                const uint32_t s = it % C::XS;
                uint8_t* dst = base + s * C::X_BYTES;
                const X* src = static_cast<const X*>(p.x) + static_cast<int64_t>(c.row0) * p.ldx +
                               kb * 128;
                const int items = c.nv * 16;  // (token, eight columns)
                for (int i0 = th; i0 < MANY_NT * 16; i0 += 64 * C::BATCH) {
                    Raw8<X> v[C::BATCH];
#pragma unroll
                    for (int b = 0; b < C::BATCH; ++b) {
                        const int i = i0 + 64 * b, o = i & 15;
                        v[b].zero();
                        if (i >= items || kb * 128 + o * 8 >= p.K) continue;
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
                        const int i = i0 + 64 * b, o = i & 15;
                        if (i >= items) continue;
                        uint4 out[C::PARTS];
                        pack_x<X>(v[b], out);
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
    } else if (warp < 8) {
        // --------------------------------------------------------- scales
        // chunks of four per row, four rows to a thread
        const int th = (tid - 192) & 63;
        const int SG = p.K / C::S;
        const int ss = p.stype == QMOE_F32 ? 4 : 2;
        const bool vec = SG % 4 == 0 && (kbeg * C::GPB) % 4 == 0 &&
                         reinterpret_cast<uintptr_t>(p.scale) % (4 * ss) == 0 &&
                         reinterpret_cast<uintptr_t>(p.zero) % 4 == 0;
        uint32_t ch = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += step) {
            const gmm::Tile c = tile_of(t);
            for (int kb = kbeg; kb < kend && ok; kb += C::CB, ++ch) {
                const int g0 = kb * C::GPB;
                uint32_t raw[4][4], zero[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = min(c.nbi * MANY_ROWS + 64 * j + th, p.N - 1);
                    const int64_t at = (static_cast<int64_t>(c.e) * p.N + n) * SG + g0;
#pragma unroll
                    for (int g = 0; g < 4; ++g) zero[j][g] = 8u;
                    if (vec && g0 + 4 <= SG) {
                        if (ss == 4) {
                            const uint4 q = __ldcg(reinterpret_cast<const uint4*>(
                                static_cast<const float*>(p.scale) + at));
                            raw[j][0] = q.x; raw[j][1] = q.y; raw[j][2] = q.z; raw[j][3] = q.w;
                        } else {
                            const uint2 q = __ldcg(reinterpret_cast<const uint2*>(
                                static_cast<const uint16_t*>(p.scale) + at));
                            raw[j][0] = q.x & 0xFFFFu; raw[j][1] = q.x >> 16;
                            raw[j][2] = q.y & 0xFFFFu; raw[j][3] = q.y >> 16;
                        }
                        if (p.zero) {
                            const uint32_t q =
                                __ldcg(reinterpret_cast<const uint32_t*>(p.zero + at));
#pragma unroll
                            for (int g = 0; g < 4; ++g) zero[j][g] = (q >> (8 * g)) & 0xFFu;
                        }
                    } else {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            raw[j][g] = g0 + g < SG ? load_raw(p.scale, at + g, p.stype) : 0u;
                            if (p.zero && g0 + g < SG) zero[j][g] = __ldcg(p.zero + at + g);
                        }
                    }
                }
                const uint32_t s = ch % C::SR;
                ok = wait(&s_empty[s], ((ch / C::SR) & 1) ^ 1);
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int at = (s * 4 + g) * MANY_ROWS + 64 * j + th;
                        sc_s[at] = typed(raw[j][g], p.stype);
                        sc_z[at] = static_cast<uint16_t>(Magic<H>::bias(zero[j][g]));
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_full[s]);
            }
        }
    } else {
        // -------------------------------------------------------- workers
        const int h = (warp - 8) >> 2, row = tid - 256;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t it = 0, na = 0, nd = 0, ch = 0;
        bool ok = true, behind = false, behind_last = false;
        gmm::Tile c = {}, cb = {};      // of the codes in hand, and of the sums behind
        float acc[MANY_NT], scale[C::GPB], scale_b[C::GPB];
        auto sums = [&]() {
#pragma unroll
            for (int g = 0; g < C::GPB; ++g) {
                const uint32_t db = nd % C::DB;
                ok = ok && wait(&d_full[h * C::DB + db], (nd / C::DB) & 1);
                if (!ok) return;
                umma::fence_after_sync();
#pragma unroll
                for (int q = 0; q < MANY_NT / 16; ++q)
                    if (16 * q < cb.np) {
                        uint32_t r[16];
                        umma::ld_32x32b_x16(tmem + lanes + (db * 2 + h) * MANY_NT + 16 * q, r);
                        umma::wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
                            gmm::fma2(acc[16 * q + i], acc[16 * q + i + 1], r[i], r[i + 1],
                                      scale_b[g], scale_b[g]);
                    }
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[h * C::DB + db]);
                ++nd;
            }
            behind = false;
            if (!behind_last) return;
            // the tile is complete
            const int n = cb.nbi * MANY_ROWS + row;
            if (ranks == 1 && n < p.N) {
#pragma unroll
                for (int i = 0; i < MANY_NT; ++i)
                    if (i < cb.nv) store_y(p, cb.row0 + i, n, acc[i] * Magic<H>::UP);
            }
        };
        for (int t = first; t < tiles && ok; t += step) {
            c = tile_of(t);
            const bool mine = live(c, h);
            for (int kb = kbeg; kb < kend; ++kb, ++it) {
                const uint32_t ws = it % C::WS, sr = ch % C::SR;
                const int kk = (kb - kbeg) % C::CB;
                if (kk == 0) ok = wait(&s_full[sr], (ch / C::SR) & 1);
                ok = ok && wait(&w_full[ws], (it / C::WS) & 1);
                if (!ok) break;
                uint4 w[4];
                const uint8_t* wr = base + C::O_W + ws * C::W_BYTES + row * 64;
                const int sw = (row >> 1) & 3;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = *reinterpret_cast<const uint4*>(wr + ((q ^ sw) << 4));
                uint32_t bias[C::GPB];
#pragma unroll
                for (int g = 0; g < C::GPB; ++g) {
                    const int at = (sr * 4 + kk * C::GPB + g) * MANY_ROWS + row;
                    scale[g] = sc_s[at];
                    bias[g] = __byte_perm(sc_z[at], 0u, 0x1010);
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&w_empty[ws]);
                    if (kk == C::CB - 1 || kb == kend - 1) mbar_arrive(&s_empty[sr]);
                }
                if (kk == C::CB - 1 || kb == kend - 1) ++ch;
                if (mine) {
                    const uint32_t ab = na % C::AB;
                    ok = wait(&a_empty[h * C::AB + ab], ((na / C::AB) & 1) ^ 1);
                    if (!ok) break;
                    umma::fence_after_sync();
                    const uint32_t a = tmem + lanes + C::TM_A + (ab * 2 + h) * 64;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t r[16];
                        const uint32_t b = bias[q * 32 / C::S];
                        codes<H>(w[q].x, b, *reinterpret_cast<uint32_t(*)[4]>(r));
                        codes<H>(w[q].y, b, *reinterpret_cast<uint32_t(*)[4]>(r + 4));
                        codes<H>(w[q].z, b, *reinterpret_cast<uint32_t(*)[4]>(r + 8));
                        codes<H>(w[q].w, b, *reinterpret_cast<uint32_t(*)[4]>(r + 12));
                        umma::st_32x32b_x16(a + 16 * q, r);
                    }
                    umma::wait_st();
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&a_full[h * C::AB + ab]);
                    ++na;
                }
                if (behind) sums();
                if (!ok) break;
                if (kb == kbeg)
#pragma unroll
                    for (int i = 0; i < MANY_NT; ++i) acc[i] = 0.f;
                behind = mine;
                behind_last = kb == kend - 1;
                cb = c;
#pragma unroll
                for (int g = 0; g < C::GPB; ++g) scale_b[g] = scale[g];
            }
        }
        if (behind && ok) sums();
        if (ranks > 1) {
            // this CTA's part of the tile, [column][weight row], where the stages were
            // (every worker is done with them); NaN if a wait ran out, so that the
            // cluster's sum does not pass for a result
            named_bar(1, 256);
            if (first < tiles)
#pragma unroll
                for (int i = 0; i < MANY_NT; ++i)
                    if (i < c.nv)
                        part[i * MANY_ROWS + row] =
                            ok ? acc[i] * Magic<H>::UP : __int_as_float(0x7FC00000);
        }
    }

    __syncwarp();
    if (ranks > 1) {
        // the ranks' parts in rank order; rank r takes columns r, r + ranks, ...
        cluster_sync();
        if (warp >= 8 && first < tiles) {
            const gmm::Tile c = tile_of(first);
            const int n = c.nbi * MANY_ROWS + tid - 256;
            for (int j = rank; j < c.nv; j += ranks) {
                const float v = gmm::cluster_sum(part + j * MANY_ROWS + tid - 256, ranks);
                if (n < p.N) store_y(p, c.row0 + j, n, v);
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
