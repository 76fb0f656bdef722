// Host build of the grouped products' tile cutting
// (moe_ffn_gb300/csrc/gmm_tiles.cuh) for the CPU tests.  Test
// infrastructure: the library does not use it.
#include <vector>

#include "../../moe_ffn_gb300/csrc/gmm_tiles.cuh"

extern "C" {

// Cuts the groups of `offsets` (E + 1 values) as the kernel does; writes up to
// cap tiles of five ints each and returns their count (-1 if over cap).
// *ok: the offsets were in order; *bound: max_tiles of the sizes.
int gmm_tiles_host(const int* offsets, int E, int M, int nt, int step, int nb, int* out, int cap, int* ok,
                   long long* bound) {
    using namespace qmoe::gmm;
    std::vector<int> lo(E), hi(E), pre(E + 1);
    *ok = 1;
    int total = 0;
    for (int e = 0; e < E; ++e) {
        if (!group_rows(offsets[e], offsets[e + 1], M, &lo[e], &hi[e])) *ok = 0;
        pre[e] = total;
        total += group_tiles(hi[e] - lo[e], nt, nb);
    }
    pre[E] = total;
    *bound = max_tiles(M, E, nt, nb);
    if (total > cap) return -1;
    for (int t = 0; t < total; ++t) {
        const Tile w = tile_at(t, nt, step, lo.data(), hi.data(), pre.data(), E);
        const int v[5] = {w.e, w.nbi, w.row0, w.nv, w.np};
        for (int i = 0; i < 5; ++i) out[5 * t + i] = v[i];
    }
    return total;
}

}
