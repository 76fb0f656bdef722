// w4.cuh — products with 4-bit weights: y[r][n] = sum_j W_g[n][j] x[r][j] for the rows
// r of group g, W[n][j] = scale[n][j / S] (code[n][j] - zero[n][j / S]), S = 32, 64 or
// 128 columns to a scale.
#pragma once
#include "gmm_tiles.cuh"
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
    int stype, xtype, ytype;
    DevCtl* err;
};

constexpr int THREADS = 256;

__device__ __forceinline__ float load_typed(const void* p, int64_t i, int type) {
    if (type == QMOE_F32) return __ldcg(static_cast<const float*>(p) + i);
    if (type == QMOE_BF16) return to_f32(ldcg_value(static_cast<const __nv_bfloat16*>(p) + i));
    return to_f32(ldcg_value(static_cast<const __half*>(p) + i));
}

// A warp per output.
__global__ void __launch_bounds__(THREADS) mm_kernel(const Params p) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    int bad = 0;
    if (p.offsets)
        for (int e = threadIdx.x; e < p.E; e += THREADS) {
            int lo, hi;
            if (!gmm::group_rows(__ldcg(p.offsets + e), __ldcg(p.offsets + e + 1), p.M, &lo, &hi))
                bad = 1;
        }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) record_error(p.err, DEV_GMM_OFFSETS);
        return;
    }
    const int64_t items = static_cast<int64_t>(p.M) * p.N;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5);
         it < items; it += step) {
        const int r = static_cast<int>(it / p.N), n = static_cast<int>(it - int64_t{r} * p.N);
        int g = 0;
        if (p.offsets) {
            if (r < __ldcg(p.offsets) || r >= __ldcg(p.offsets + p.E)) continue;
            int hi = p.E;  // the last group that starts at or before r
            while (hi - g > 1) {
                const int mid = (g + hi) / 2;
                if (__ldcg(p.offsets + mid) <= r) g = mid;
                else hi = mid;
            }
        }
        const int64_t row = static_cast<int64_t>(g) * p.N + n;
        const uint8_t* w = p.W + row * (p.K / 2);
        const int64_t s0 = row * (p.K / p.S), x0 = static_cast<int64_t>(r) * p.ldx;
        float sum = 0.f;
        for (int j = lane * 2; j < p.K; j += 64) {
            const int b = __ldcg(w + j / 2);
            const int64_t s = s0 + j / p.S;
            const int z = p.zero ? __ldcg(p.zero + s) & 15 : 8;
            const float a = static_cast<float>((b & 15) - z) * load_typed(p.x, x0 + j, p.xtype);
            const float c = fmaf(static_cast<float>((b >> 4) - z),
                                 load_typed(p.x, x0 + j + 1, p.xtype), a);
            sum = fmaf(load_typed(p.scale, s, p.stype), c, sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            const int64_t at = static_cast<int64_t>(r) * p.ldy + n;
            if (p.ytype == QMOE_F32) static_cast<float*>(p.y)[at] = sum;
            else if (p.ytype == QMOE_BF16)
                static_cast<__nv_bfloat16*>(p.y)[at] = from_f32<__nv_bfloat16>(sum);
            else static_cast<__half*>(p.y)[at] = from_f32<__half>(sum);
        }
    }
}

}  // namespace w4
}  // namespace qmoe
