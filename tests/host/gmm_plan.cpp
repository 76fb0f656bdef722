// Host build of the rule by which the grouped products choose their kernel, and of
// the cut of one group (moe_ffn_gb300/csrc/gmm_tiles.cuh).  Test infrastructure:
// the library does not use it.
#include "../../moe_ffn_gb300/csrc/gmm_tiles.cuh"

extern "C" {

int token_tile_host(long long M, int E, int grouped, int nb, int f8, int swiglu, int sms) {
    return qmoe::gmm::token_tile(M, E, grouped != 0, nb, f8 != 0, swiglu != 0, sms);
}

long long max_tiles_host(long long M, int E, int nt, int nb) {
    return qmoe::gmm::max_tiles(M, E, nt, nb);
}

int group_of_host(int t, const int* pre, int E) {
    return qmoe::gmm::group_of(E, [&](int e0) {
        int n = 0;
        for (int i = e0; i < e0 + 32 && i < E; ++i) n += pre[i] <= t;
        return n;
    });
}

}
