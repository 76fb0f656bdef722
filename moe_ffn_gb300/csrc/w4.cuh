// w4.cuh — products with 4-bit weights: y[r][n] = sum_j W_g[n][j] x[r][j] for the rows
// r of group g, W[n][j] = scale[n][j / S] (code[n][j] - zero[n][j / S]), S = 32, 64 or
// 128 columns to a scale.
//
// The codes minus their zero point are integers of -15..15, exact in 16 bits, so the
// tensor core multiplies them by x exactly; the sum over the columns of one scale comes
// from it in f32, and is multiplied by the scale and added up in f32.  An f32 x is cut
// into three bf16 values that add up to it (8 significant bits each), which take three
// columns of the product and are added at the end.
//
// Orientation: weight rows are the product's M side, token rows its N side.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gmm.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace qmoe {
namespace w4 {

struct Params {
    const uint8_t* W;       // [E][N][K / 2], the even column in the low half of a byte
    const void* scale;      // [E][N][K / S]
    const uint8_t* zero;    // [E][N][K / S], or null: 8 everywhere
    const void* x;          // [M][K], rows ldx apart
    void* y;                // [M][N], rows ldy apart
    const int32_t* offsets; // [E + 1], or null: one group of all rows
    int64_t ldx, ldy;
    int M, N, K, E, S;
    int stype, ytype;
    int vec_x;              // rows of x are whole aligned 16-byte units
    int nb;                 // tiles of W
    int tiles;              // of the call, without offsets
    int nt;                 // tokens of a tile
    int cols;               // columns that the tokens of a tile take in shared memory
    int wk, rts_log;        // parts of K among a CTA's warps; 2^rts_log = 8 / wk row tiles
    int rank_units;         // 128-column units of K of a CTA of a cluster
    int pass_rounds;        // rounds of its blocks whose x is in shared memory at a time
    int slot;               // outputs of a tile, or 0 without a cluster
    DevCtl* err;
};

// A barrier over the cluster's threads, in two steps, that orders no memory.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A store to the address that `p` has in CTA `rank`'s shared memory.
__device__ __forceinline__ void cluster_st_f32(float* p, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "f"(v) : "memory");
}

// A scale as f32.  The formula multiplies every weight by it, so an infinite one makes
// infinities of both signs or NaN (a code at its zero point) of them, and NaN of their sum;
// here it meets the sum (for an f32 x those of its three parts), so it is taken as NaN.
__device__ __forceinline__ float scale_value(uint32_t raw, int type) {
    const float s = type == QMOE_F32    ? __uint_as_float(raw)
                    : type == QMOE_BF16 ? __uint_as_float(raw << 16)
                                        : __half2float(__ushort_as_half(static_cast<unsigned short>(raw)));
    return fmaf(s, 0.f, s);
}
__device__ __forceinline__ uint32_t load_raw(const void* p, int64_t i, int type) {
    return type == QMOE_F32 ? __ldcg(static_cast<const unsigned*>(p) + i)
                            : __ldcg(static_cast<const unsigned short*>(p) + i);
}

__device__ __forceinline__ void store_y(const Params& p, int64_t r, int n, float v) {
    const int64_t at = r * p.ldy + n;
    if (p.ytype == QMOE_F32) static_cast<float*>(p.y)[at] = v;
    else if (p.ytype == QMOE_BF16)
        static_cast<__nv_bfloat16*>(p.y)[at] = from_f32<__nv_bfloat16>(v);
    else static_cast<__half*>(p.y)[at] = from_f32<__half>(v);
}

// Weight row n of a tile's tokens.
template <int NT>
__device__ __forceinline__ void store_column(const Params& p, const gmm::Tile& c, int n,
                                             const float (&v)[NT], float up) {
    const int64_t at = static_cast<int64_t>(c.row0) * p.ldy + n;
    if (p.ytype == QMOE_F32) {
        float* y = static_cast<float*>(p.y) + at;
#pragma unroll
        for (int i = 0; i < NT; ++i, y += p.ldy)
            if (i < c.nv) *y = v[i] * up;
    } else if (p.ytype == QMOE_BF16) {
        __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + at;
#pragma unroll
        for (int i = 0; i < NT; ++i, y += p.ldy)
            if (i < c.nv) *y = from_f32<__nv_bfloat16>(v[i] * up);
    } else {
        __half* y = static_cast<__half*>(p.y) + at;
#pragma unroll
        for (int i = 0; i < NT; ++i, y += p.ldy)
            if (i < c.nv) *y = from_f32<__half>(v[i] * up);
    }
}

template <class X>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<X, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <class X>
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<X, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes to 16-bit values, exactly.  The bits of a code at the low end of a 16-bit float
// are a subnormal: code 2^-24 (f16) or code 2^-133 (bf16; the encoding stays linear over
// the first eight bits).  One fused multiplication by a power of two brings it into the
// normal range and takes the zero point from it: (code - zero) / UP, so that a word of
// eight codes costs one shift, four ANDs and four of these.  UP comes back in the end.
template <class X>
struct Magic {
    static constexpr bool F16 = std::is_same<X, __half>::value;
    static constexpr float UP = F16 ? 512.f : 64.f;
    // multipliers of codes in bits 0..3 and 4..7 of a half: 2^15, 2^11 or 2^127, 2^123
    static constexpr uint32_t LOW = F16 ? 0x78007800u : 0x7F007F00u;
    static constexpr uint32_t HIGH = F16 ? 0x68006800u : 0x7D007D00u;
    // -zero / UP, twice
    static __device__ __forceinline__ uint32_t bias(uint32_t zero) {
        const float v = static_cast<float>(zero & 15u) * (-1.f / UP);
        return F16 ? pack_f16(v, v) : pack_bf16(v, v);
    }
};
template <class X>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (Magic<X>::F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// A word of eight codes: a[i] holds codes i and i + 4.
template <class X>
__device__ __forceinline__ void codes(uint32_t w, uint32_t bias, uint32_t (&a)[4]) {
    const uint32_t v = w >> 8;
    a[0] = fma2<X>(w & 0x000F000Fu, Magic<X>::LOW, bias);
    a[1] = fma2<X>(w & 0x00F000F0u, Magic<X>::HIGH, bias);
    a[2] = fma2<X>(v & 0x000F000Fu, Magic<X>::LOW, bias);
    a[3] = fma2<X>(v & 0x00F000F0u, Magic<X>::HIGH, bias);
}

// Eight f32 values in three bf16 parts each, of eight leading bits, cut off one after
// another, which leaves exact rests: the upper halves of h.  (Infinities and NaN have no
// rest: they stay whole in part 0.)
__device__ __forceinline__ void split3(const Raw8<float>& v, uint32_t (&h)[3][8]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float f1 = __uint_as_float(v.w[e]) - __uint_as_float(v.w[e] & 0xFFFF0000u);
        const float f2 = f1 - __uint_as_float(__float_as_uint(f1) & 0xFFFF0000u);
        h[0][e] = v.w[e];
        h[1][e] = __float_as_uint(f1);
        h[2][e] = __float_as_uint(f2);
        top = max(top, v.w[e] & 0x7FFFFFFFu);
    }
    if (top < 0x7F800000u) return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if ((v.w[e] & 0x7F800000u) == 0x7F800000u) {
            if (v.w[e] & 0x7FFFFFu) h[0][e] |= 0x00400000u;  // (a NaN by its low bits alone)
            h[1][e] = h[2][e] = 0u;
        }
}
// The bf16 in the upper halves of two words, a's first.
__device__ __forceinline__ uint32_t upper2(uint32_t a, uint32_t b) {
    return __byte_perm(a, b, 0x7632);
}
// Eight values of x as pairs (0,4) (1,5) (2,6) (3,7), the order in which codes() leaves a
// word; an f32 x in three parts.
template <class X>
__device__ __forceinline__ void pack_x(const Raw8<X>& v,
                                       uint4 (&out)[std::is_same<X, float>::value ? 3 : 1]) {
    if constexpr (std::is_same<X, float>::value) {
        uint32_t h[3][8];
        split3(v, h);
#pragma unroll
        for (int q = 0; q < 3; ++q)
            out[q] = make_uint4(upper2(h[q][0], h[q][4]), upper2(h[q][1], h[q][5]),
                                upper2(h[q][2], h[q][6]), upper2(h[q][3], h[q][7]));
    } else {
        out[0] = make_uint4(__byte_perm(v.w[0], v.w[2], 0x5410), __byte_perm(v.w[0], v.w[2], 0x7632),
                            __byte_perm(v.w[1], v.w[3], 0x5410), __byte_perm(v.w[1], v.w[3], 0x7632));
    }
}

// ------------------------------------------------------- few rows per group
// The eight warps of a CTA are WK parts of its K range times 8 / WK tiles of 16 weight
// rows, by 8 NB columns of x.  A warp takes K in blocks of four units of 128 columns,
// the next block's 16-byte loads in flight while this one's codes are multiplied; the
// parts are added through shared memory in warp order, those of a cluster's CTAs, which
// share K where there are few tiles, in rank order.
// A lane loads the 32 codes that it multiplies from one row straight to registers, and
// which columns the MMA's k positions stand for is chosen to fit: x lies in shared
// memory in that order.  The columns of one scale have to be one MMA's k range: for S =
// 128 the four lanes of a row hold 32 columns each; for 64 and 32 they first exchange
// words.
//
// No pipe is full (14336 x 4096, five rows: issue 54%, ALU 44%, tensor 11%, DRAM 23%).  A unit
// (32 codes a lane, 8 MMAs) takes a scheduler 158 clocks in a probe of the loop alone, which
// makes about half of a call; the other half, starts, tile changes and sums, was not
// measured apart.  Measured: 14336 x 4096, one row
// 10.9 us (2.8 TB/s), five rows 12.7; 4096 x 4096, one row 5.5 us cold (by clock stamps
// about 2 us before the first product, 1.3 for the products, 0.4 for the sum); eight
// groups of one row, 768 x 2048 5.6 us.  With three shifts and four subtractions a word
// of codes, and a table of groups where there are none, 14336 x 4096 took one row 13.4 us.
constexpr int WARPS = 8;
constexpr int THREADS = 32 * WARPS;
constexpr int UNIT = 128;
constexpr int BLOCK = 4;      // units of a block
constexpr int MAX_RANKS = 8;
constexpr int RED_LD = 20;    // 16 rows of a column, padded: conflict-free

// The unit's place of its o-th group of eight columns: step j, lane t of the quad.
template <int S>
__device__ __forceinline__ void place(int o, int* j, int* t) {
    if (S == 128) { *t = o >> 2; *j = o & 3; }
    else if (S == 64) { *j = ((o >> 3) << 1) | (o & 1); *t = ((o >> 2) & 1) | (o & 2); }
    else { *j = o >> 2; *t = o & 3; }
}

// Words (one per step j) of a row after the quad's exchange.
template <int S>
__device__ __forceinline__ void exchange(uint4& v, int t) {
    if constexpr (S < 128) {  // lanes t and t ^ 2
        const bool hi = t & 2;
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, hi ? v.x : v.z, 2);
        const uint32_t r1 = __shfl_xor_sync(0xffffffffu, hi ? v.y : v.w, 2);
        if (hi) { v.x = r0; v.y = r1; } else { v.z = r0; v.w = r1; }
    }
    if constexpr (S == 32) {  // lanes t and t ^ 1
        const bool odd = t & 1;
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1);
        const uint32_t r1 = __shfl_xor_sync(0xffffffffu, odd ? v.z : v.w, 1);
        if (odd) { v.x = r0; v.z = r1; } else { v.y = r0; v.w = r1; }
    }
}

// Bytes of shared memory before x: the tiles' table, the warps' parts, and those of
// the ranks (`slots` values in all).
__host__ __device__ constexpr int few_fixed(int E, int nb_cols, int slots) {
    return ((3 * E + 1) * 4 + 15) / 16 * 16 + 2 * WARPS * 8 * nb_cols * RED_LD * 4 +
           slots * 2 * 4;
}

template <class X, int S, int NB>
__global__ void __launch_bounds__(THREADS, 2) few_kernel(const Params p) {
    constexpr bool F32X = std::is_same<X, float>::value;
    constexpr int PARTS = F32X ? 3 : 1;
    constexpr int NS = UNIT / S;  // scales of a unit
    using H = typename std::conditional<std::is_same<X, __half>::value, __half,
                                        __nv_bfloat16>::type;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    const int lg = 31 - __clz(ranks);
    const int cluster = blockIdx.x >> lg, clusters = gridDim.x >> lg;
    const int kw = warp >> p.rts_log, rts = 1 << p.rts_log, rt = warp & (rts - 1);
    int* t_lo = reinterpret_cast<int*>(smem);
    int* t_hi = t_lo + p.E;
    int* t_pre = t_hi + p.E;
    float* red = reinterpret_cast<float*>(smem + ((3 * p.E + 1) * 4 + 15) / 16 * 16);
    float* far = red + 2 * WARPS * 8 * NB * RED_LD;
    uint4* xs = reinterpret_cast<uint4*>(smem + few_fixed(p.E, NB, p.slot * ranks));
    int tiles = p.tiles;
    const int units = (p.K + UNIT - 1) / UNIT;
    const int ub = min(rank * p.rank_units, units), ue = min(ub + p.rank_units, units);
    const int SG = p.K / S;  // scales of a row
    // rounds: a block to each of the wk parts
    const int kw_shift = 5 - p.rts_log;  // log2 of the units of a round, 4 wk
    static_assert(WARPS * BLOCK == 32, "kw_shift");
    const int rounds = max(1, (ue - ub + (1 << kw_shift) - 1) >> kw_shift);

    // what is loaded: rounds of the tile `next`
    uint4 w[BLOCK][2];                     // rows g and g + 8
    uint32_t s_raw[2][NS], z_raw[2][NS];   // of the block's unit t
    gmm::Tile next;
    const uint8_t* l_w[2];
    int64_t l_s[2];
    auto look_up = [&](int tile) {
        if (p.offsets) {
            next = gmm::tile_at_warp(tile, p.nt, 1, t_lo, t_hi, t_pre, p.E);
        } else {
            const int lo = 0, hi = p.M;
            next = gmm::tile_in(0, tile, p.nt, 1, &lo, &hi, &lo);
        }
        const int64_t base = static_cast<int64_t>(next.e) * p.N;
        const int n = (next.nbi * rts + rt) * 16 + g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t r = base + min(n + 8 * h, p.N - 1);
            l_w[h] = p.W + r * (p.K / 2) + t * 16;
            l_s[h] = r * SG;
        }
    };
    // (what does not depend on earlier launches comes before the wait for them)
    if (!p.offsets) look_up(cluster);
    // All CTAs of the cluster run from here on, so that their shared memory may be written.
    // (In this place it costs a call at most 1%; split in two, or in the tiles' loop before
    // the first store, it cost calls without clusters too 1 to 6%, by another allocation of
    // registers.)
    if (ranks > 1) {
        cluster_arrive();
        cluster_wait();
    }
    pdl_wait();
    pdl_trigger();
    if (p.offsets) {
        gmm::build_tables(p, p.nt, p.nb, t_lo, t_hi, t_pre);
        tiles = t_pre[p.E];
        if (cluster >= tiles) return;
    }
    // the first unit of this warp's block of a round, and whether the block is whole
    auto block_at = [&](int round) { return ub + (round << kw_shift) + kw * BLOCK; };
    auto whole = [&](int u) { return u + BLOCK <= ue && (u + BLOCK) * UNIT <= p.K; };
    auto load_unit = [&](int u, bool all, int i) {
        if (all) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[i][h] = __ldcg(reinterpret_cast<const uint4*>(l_w[h] + u * (UNIT / 2)) +
                                 i * (UNIT / 32));
        } else {
            const bool in = u + i < ue && (u + i) * UNIT + t * 32 < p.K;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[i][h] = in ? __ldcg(reinterpret_cast<const uint4*>(l_w[h] + (u + i) * (UNIT / 2)))
                             : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_scales = [&](int u, bool all) {
        const int gi = (u + t) * NS;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NS; ++j) {
                const bool in = all || (u + t < ue && gi + j < SG);
                s_raw[h][j] = 0u;
                z_raw[h][j] = 8u;
                if (in) s_raw[h][j] = load_raw(p.scale, l_s[h] + gi + j, p.stype);
                if (in && p.zero) z_raw[h][j] = __ldcg(p.zero + l_s[h] + gi + j);
            }
    };

    float sc[2][NS];      // of the block in hand, unit t
    uint32_t zb[2][NS];
    float acc[NB][4];
    int at_col[NB];       // this lane's columns of x (one that exists where its own does not)
    const int js = p.cols * 4;
    auto product = [&](int i, const uint4* xu) {
        uint4 v[2] = {w[i][0], w[i][1]};
        exchange<S>(v[0], t);
        exchange<S>(v[1], t);
        const int src = (lane & ~3) | i;
        constexpr int PER = S / 32;  // steps of a scale
        float d[NB][4];
        uint32_t bias[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t c = j == 0 ? v[h].x : j == 1 ? v[h].y : j == 2 ? v[h].z : v[h].w;
                if (j % PER == 0) bias[h] = __shfl_sync(0xffffffffu, zb[h][j / PER], src);
                codes<H>(c, bias[h], a[h]);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint4 b = xu[j * js + at_col[n]];
                if (j % PER == 0) mma16_first<H>(d[n], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                else mma16<H>(d[n], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                mma16<H>(d[n], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
            }
            if (j % PER == PER - 1) {
                const float s0 = __shfl_sync(0xffffffffu, sc[0][j / PER], src);
                const float s8 = __shfl_sync(0xffffffffu, sc[1][j / PER], src);
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    acc[n][0] = fmaf(s0, d[n][0], acc[n][0]);
                    acc[n][1] = fmaf(s0, d[n][1], acc[n][1]);
                    acc[n][2] = fmaf(s8, d[n][2], acc[n][2]);
                    acc[n][3] = fmaf(s8, d[n][3], acc[n][3]);
                }
            }
        }
    };
    // x of some rounds, in the order in which the products take it: for unit, step j,
    // column and lane t, the eight values of its place as pairs (0,4) (1,5) (2,6) (3,7)
    // `then` runs once, behind the first loads.
    auto stage_x = [&](int row0, int nv, int round, auto then) {
        const int u0 = ub + (round << kw_shift);
        const int n8 = min(p.pass_rounds << kw_shift, ue - u0) * 16;  // eights of columns
        constexpr int AHEAD = F32X ? 2 : 4;  // loads in flight per thread
        int tok = 0, o = tid;
        auto settle = [&]() {
            while (o >= n8 && tok < nv) {
                o -= n8;
                ++tok;
            }
        };
        settle();
        bool first = true;
        do {
            Raw8<X> v[AHEAD];
            int at[AHEAD];  // token and eight of columns
#pragma unroll
            for (int b = 0; b < AHEAD; ++b) {
                at[b] = -1;
                if (tok >= nv) continue;
                at[b] = tok << 24 | o;
                const int c = u0 * UNIT + o * 8;
                const X* src = static_cast<const X*>(p.x) + (row0 + tok) * p.ldx + c;
                if (c >= p.K) v[b].zero();
                else if (p.vec_x) v[b].load(src);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const X one = ldcg_value(src + e);
                        if constexpr (F32X) v[b].w[e] = __float_as_uint(one);
                        else reinterpret_cast<X*>(v[b].w)[e] = one;
                    }
                o += THREADS;
                settle();
            }
            if (first) then();
            first = false;
#pragma unroll
            for (int b = 0; b < AHEAD; ++b) {
                if (at[b] < 0) continue;
                const int ob = at[b] & 0xFFFFFF;
                int j, tt;
                place<S>(ob & 15, &j, &tt);
                uint4* dst = xs + static_cast<int64_t>((ob >> 4) * 4 + j) * js +
                             (at[b] >> 24) * PARTS * 4 + tt;
                uint4 out[PARTS];
                pack_x<X>(v[b], out);
#pragma unroll
                for (int q = 0; q < PARTS; ++q) dst[q * 4] = out[q];
            }
        } while (tok < nv);
    };

    if (p.offsets) look_up(cluster);
    auto load_first = [&]() {
        const int u = block_at(0);
        const bool all = whole(u);
        load_scales(u, all);
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) load_unit(u, all, i);
    };
    int staged = -1, buf = 0;  // -1: nothing is loaded yet
    for (int tile = cluster; tile < tiles; tile += clusters) {
        const gmm::Tile c = next;
        const bool more = tile + clusters < tiles;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            at_col[n] = min(n * 8 + g, c.nv * PARTS - 1) * 4 + t;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
        }
        int in_pass = 0;
        for (int round = 0; round < rounds; ++round) {
            if (in_pass == 0 && (p.pass_rounds < rounds || staged != c.row0)) {
                if (round > 0) __syncthreads();  // (a tile ends with a barrier)
                // (the first tile's x, which comes from L2, and its codes, from further
                // away, are asked for at once)
                stage_x(c.row0, c.nv, round, [&]() {
                    if (staged < 0) load_first();
                });
                staged = c.row0;
                __syncthreads();
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NS; ++j) {
                    sc[h][j] = scale_value(s_raw[h][j], p.stype);
                    zb[h][j] = Magic<H>::bias(z_raw[h][j]);
                }
            const bool last = round + 1 == rounds;
            if (last && more) look_up(tile + clusters);
            const bool load = !last || more;
            const int u = block_at(last ? 0 : round + 1);
            const bool all = whole(u);
            if (load) load_scales(u, all);
            const int left = ue - block_at(round);  // units of this block and after it
            const uint4* xu = xs + ((in_pass << kw_shift) + kw * BLOCK) * 4 * js;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) {
                if (i < left) product(i, xu + i * 4 * js);
                if (load) load_unit(u, all, i);
            }
            if (++in_pass == p.pass_rounds) in_pass = 0;
        }
        // the warps' parts, in order (two buffers: one barrier a tile)
        float* mine = red + (buf * WARPS + warp) * 8 * NB * RED_LD;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float* at = mine + (n * 8 + 2 * t) * RED_LD + g;
            at[0] = acc[n][0] * Magic<H>::UP;
            at[RED_LD] = acc[n][1] * Magic<H>::UP;
            at[8] = acc[n][2] * Magic<H>::UP;
            at[RED_LD + 8] = acc[n][3] * Magic<H>::UP;
        }
        __syncthreads();
        const int shift = 4 + p.rts_log, rows16 = 16 << p.rts_log;
        for (int i = tid; i < rows16 * c.nv; i += THREADS) {
            const int row = i & (rows16 - 1), tok = i >> shift;
            const float* at = red + ((buf * WARPS + (row >> 4)) * 8 * NB + tok * PARTS) * RED_LD + (row & 15);
            float v = 0.f;
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part) {
                float q[WARPS];
#pragma unroll
                for (int k = 0; k < WARPS; ++k)
                    q[k] = k < p.wk ? at[((k << p.rts_log) * 8 * NB + part) * RED_LD] : 0.f;
#pragma unroll
                for (int k = 0; k < WARPS; ++k) v += q[k];
            }
            const int n = c.nbi * rows16 + row;
            if (ranks > 1) cluster_st_f32(far + (buf * ranks + rank) * p.slot + i, 0u, v);
            else if (n < p.N) store_y(p, c.row0 + tok, n, v);
        }
        if (ranks > 1) {
            cluster_sync();
            if (rank == 0)
                for (int i = tid; i < rows16 * c.nv; i += THREADS) {
                    const int n = c.nbi * rows16 + (i & (rows16 - 1));
                    float v = 0.f;
                    for (int k = 0; k < ranks; ++k) v += far[(buf * ranks + k) * p.slot + i];
                    if (n < p.N) store_y(p, c.row0 + (i >> shift), n, v);
                }
        }
        buf ^= 1;
    }
}

}  // namespace w4
}  // namespace qmoe
