// Host build of the choice between the 4-bit products' kernels
// (moe_ffn_gb300/csrc/w4_rule.cuh).  Test infrastructure: the library does not use it.
#include "../../moe_ffn_gb300/csrc/w4_rule.cuh"

extern "C" int many_rows_host(long long M, int E, long long N, long long K, int f32) {
    return qmoe::w4::many_rows(M, E, N, K, f32 != 0);
}
