// gmm_tiles.cuh — how the grouped products cut their work into tiles, and which
// kernel takes a call.  Compiled for the host as well, so that both can be checked
// on a CPU.
#pragma once
#include <cstdint>

#include "route.cuh"  // QMOE_HD

namespace qmoe {
namespace gmm {

// One tile: group e, weight tile nbi, token rows row0 .. row0 + nv - 1.
struct Tile {
    int e, nbi, row0, nv, np;  // np: nv rounded up to `step`
};

// A group's rows [*lo, *hi) from its two offsets, clamped so that
// 0 <= *lo <= *hi <= M whatever they hold; true if they were in order.
QMOE_HD bool group_rows(int lo, int hi, int M, int* lo_out, int* hi_out) {
    const bool ok = lo >= 0 && hi >= lo && hi <= M;
    lo = lo < 0 ? 0 : lo > M ? M : lo;
    hi = hi < lo ? lo : hi > M ? M : hi;
    *lo_out = lo;
    *hi_out = hi;
    return ok;
}

// Tiles of a group of `rows` rows: token tiles of at most nt rows times nb
// weight tiles.
QMOE_HD int group_tiles(int rows, int nt, int nb) {
    return static_cast<int>((static_cast<int64_t>(rows) + nt - 1) / nt) * nb;
}

// Tile t, 0 <= t < pre[E]: lo, hi the groups' rows, pre[e] the tiles of the
// groups before e.  A group of more than nt rows is cut into c = ceil(rows / nt)
// token tiles of ceil(rows / c) rows rounded up to `step`, the last the rest of
// them (it may be short: 193 rows by 96 in steps of 32 are 96 + 96 + 1).  step is
// a power of two that divides nt, the MMA's N step: 16, or 32 for a CTA pair.  The
// token tiles of one weight tile are consecutive, so CTAs at work at the same time
// share the weight tile in L2.
QMOE_HD Tile tile_in(int a, int t, int nt, int step, const int* lo, const int* hi,
                     const int* pre) {
    Tile r;
    r.e = a;
    const int rows = hi[a] - lo[a];
    const int local = t - pre[a];
    int ts = nt;
    r.nbi = local;
    r.row0 = lo[a];
    if (rows > nt) {  // (the divisions only where a group has several token tiles)
        const unsigned c = static_cast<unsigned>(rows - 1) / nt + 1;
        ts = static_cast<int>((static_cast<unsigned>(rows - 1) / c + step) & ~(step - 1));
        r.nbi = static_cast<int>(static_cast<unsigned>(local) / c);
        r.row0 += (local - r.nbi * static_cast<int>(c)) * ts;
    }
    r.nv = hi[a] - r.row0 < ts ? hi[a] - r.row0 : ts;
    r.np = (r.nv + step - 1) & ~(step - 1);
    return r;
}
// The last group a with pre[a] <= t, 32 groups at a step; count(e0) is the number
// of them among e0 .. e0 + 31 (below E).
template <class Count>
QMOE_HD int group_of(int E, Count count) {
    int a = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int n = count(e0);
        a += n;
        if (n < 32) break;
    }
    return a - 1;
}
#if defined(__CUDACC__)
// Tile t by a whole warp: a ballot per step (a bisection's seven dependent loads
// took a tenth of a short tile's time).
__device__ __forceinline__ Tile tile_at_warp(int t, int nt, int step, const int* lo,
                                             const int* hi, const int* pre, int E) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    const int a = group_of(E, [&](int e0) {
        return __popc(__ballot_sync(0xffffffffu, e0 + lane < E && pre[e0 + lane] <= t));
    });
    return tile_in(a, t, nt, step, lo, hi, pre);
}
#else
// The same for the host, the warp's lanes one after another.
QMOE_HD Tile tile_at(int t, int nt, int step, const int* lo, const int* hi, const int* pre, int E) {
    const int a = group_of(E, [&](int e0) {
        int n = 0;
        for (int lane = 0; lane < 32; ++lane) n += e0 + lane < E && pre[e0 + lane] <= t;
        return n;
    });
    return tile_in(a, t, nt, step, lo, hi, pre);
}
#endif

// Most tiles that M rows in E groups can make: sum of ceil(r / nt) over at most
// min(M, E) groups that have rows, each at most (r + nt - 1) / nt.
QMOE_HD int64_t max_tiles(int64_t M, int E, int nt, int nb) {
    const int64_t groups = M < E ? M : E;
    return (M + groups * (nt - 1)) / nt * nb;
}

// Columns (token rows) of the tiles of the kernel that a call takes: FEW_ROWS for
// the kernel of small tiles, else the CTA pairs' 128 or 192 (e4m3), 128 or 256
// (16-bit types), 96 (SwiGLU form).
constexpr int FEW_ROWS = 32;

// The kernel for few rows: up to 16 rows per group, where its tile of 32 columns
// holds most groups (32 without groups), and beyond that as long as its small tiles
// still fit the SMs at once, for the other kernel's 256-row tiles then leave most
// of them idle.  e4m3, this kernel against the pair kernel: 2048 x 2048, 33 / 256
// rows 6.2 / 8.2 us against 9.5 / 12.2; 4096 x 4096 (32 row tiles), 128 rows 12.5
// against 16.4; 64 groups, 1024 x 2048, 16 rows each 28.7 against 30.5, 64 rows
// each 41.7 against 32.4.
QMOE_HD bool few_rows(int64_t M, int E, bool grouped, int nb, int sms) {
    const int64_t groups = M < E ? M : E;
    return M <= (grouped ? 16 * groups : 32) || max_tiles(M, E, FEW_ROWS, nb) <= sms;
}

// Whether the pair kernel takes its narrow tiles (128 columns) or the wide ones
// (192 for e4m3, 256 for 16-bit types), which do more work per byte but may leave
// pairs idle.
//   Narrow tiles that all fit the pairs at once: always (one pass either way).
//     4096 x 4096, e4m3, 256 / 512 rows: 16.8 / 17.5 us against 19.2 / 21.6; bf16
//     20.8 / 21.6 against 24.9 / 25.1.
//   e4m3, one group: a pass of narrow tiles takes 3/4 of one of wide tiles.
//     4096 x 4096, 640 / 1024 rows (2 passes against 1 / 2 against 2): 30.0 / 30.4
//     against 20.6 / 39.4; 14336 x 4096, 1024 / 1536 rows (6 against 5 / 9 against
//     6): 82.6 / 121 against 92 / 110.
//   e4m3, more groups, whose sizes only the device knows: up to 128 rows per
//     group on average.  64 groups, 1024 x 2048, 64 / 128 / 192 rows each: 32.4 /
//     37.0 / 51.5 against 33.5 / 41.4 / 47.2.  (Not every shape above 128 gains: 8
//     groups of 256 rows, 2048 x 2048, two tiles either way: 19.3 against 22.0.)
QMOE_HD bool narrow_tiles(int64_t M, int E, int nb, bool f8, int sms) {
    const int pair_nb = (nb + 1) / 2, pairs = sms / 2;
    const int64_t narrow = max_tiles(M, E, 128, pair_nb);
    if (narrow <= pairs) return true;
    if (!f8) return false;
    if (E > 1) return M <= int64_t{128} * (M < E ? M : E);
    const int64_t wide = max_tiles(M, 1, 192, pair_nb);
    return 3 * ((narrow + pairs - 1) / pairs) < 4 * ((wide + pairs - 1) / pairs);
}

QMOE_HD int token_tile(int64_t M, int E, bool grouped, int nb, bool f8, bool swiglu, int sms) {
    if (few_rows(M, E, grouped, nb, sms)) return FEW_ROWS;
    if (swiglu) return 96;
    return narrow_tiles(M, E, nb, f8, sms) ? 128 : f8 ? 192 : 256;
}

}  // namespace gmm
}  // namespace qmoe
