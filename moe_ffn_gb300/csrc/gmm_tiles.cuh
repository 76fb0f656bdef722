// gmm_tiles.cuh — how the grouped products cut their work into tiles.
// Compiled for the host as well, so the cutting can be checked on a CPU.
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
// groups before e.  A group is cut into ceil(rows / nt) token tiles of nearly
// equal size (multiples of `step`, a power of two that divides nt; the MMA's
// N step: 16, or 32 for a CTA pair); the token tiles of one weight
// tile are consecutive, so CTAs at work at the same time share the weight
// tile in L2.
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
#if defined(__CUDACC__)
// Tile t, its group found by a whole warp, 32 groups at a step: the last a with
// pre[a] <= t (a bisection's seven dependent loads took a tenth of a short tile's time).
__device__ __forceinline__ Tile tile_at_warp(int t, int nt, int step, const int* lo,
                                             const int* hi, const int* pre, int E) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int a = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int n = __popc(__ballot_sync(0xffffffffu, e0 + lane < E && pre[e0 + lane] <= t));
        a += n;
        if (n < 32) break;
    }
    return tile_in(a - 1, t, nt, step, lo, hi, pre);
}
#else
// The same for the host, by bisection: pre[a] <= t < pre[a + 1].
QMOE_HD Tile tile_at(int t, int nt, int step, const int* lo, const int* hi, const int* pre, int E) {
    int a = 0, b = E;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (pre[m] <= t) a = m; else b = m;
    }
    return tile_in(a, t, nt, step, lo, hi, pre);
}
#endif

// Most tiles that M rows in E groups can make: sum of ceil(r / nt) over at most
// min(M, E) groups that have rows, each at most (r + nt - 1) / nt.
QMOE_HD int64_t max_tiles(int64_t M, int E, int nt, int nb) {
    const int64_t groups = M < E ? M : E;
    return (M + groups * (nt - 1)) / nt * nb;
}

}  // namespace gmm
}  // namespace qmoe
