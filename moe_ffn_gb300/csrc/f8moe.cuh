// f8moe.cuh — the kernels around the e4m3 products: quantising rows, sorting
// a layer's (token, slot) pairs by expert, and adding the experts' outputs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "f8.cuh"
#include "gmm.cuh"
#include "ptx.cuh"

namespace qmoe {
namespace f8 {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// ---------------------------------------------------------------- quantise
// Sixteen lanes share a 128-column block, eight consecutive columns each:
// one or two 16-byte loads, a four-step maximum, one 8-byte store.  Bound by
// HBM: (size + 1) bytes per element.  VEC needs 16-byte aligned rows and
// whole groups of eight columns; the other form loads element by element.
//
// With pos (the MoE layer), row t is token t and its codes go to the rows
// pos[t * k + s] of q, one for each slot that names an expert.
struct QuantParams {
    const void* x;
    int64_t ldx;
    uint8_t* q;       // [rows][cols]
    float* s;         // [rows][nblk]
    const int32_t* pos;
    int k;            // slots per token (pos)
    int64_t rows;
    int cols, nblk;
};
constexpr int Q_THREADS = 256;

template <class T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src));
        const float4 b = __ldcg(reinterpret_cast<const float4*>(src) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = __ldcg(reinterpret_cast<const uint4*>(src));
        const T* h = reinterpret_cast<const T*>(&a);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(h[i]);
    }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(const QuantParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * Q_THREADS + threadIdx.x) >> 4;
    const int sub = threadIdx.x & 15;
    const bool live = item < p.rows * p.nblk;
    const int64_t row = live ? item / p.nblk : 0;
    const int blk = live ? static_cast<int>(item - row * p.nblk) : 0;
    const int c0 = blk * F8_BLOCK + sub * 8;
    const T* src = static_cast<const T*>(p.x) + row * p.ldx + c0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (live) {
        if constexpr (VEC) {
            if (c0 < p.cols) load8(src, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i < p.cols) v[i] = to_f32(src[i]);
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_abs_bits(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!live) return;
    float s, inv;
    f8_scale(m, &s, &inv);
    uint2 q;
    q.x = f8_pack2(v[0] * inv, v[1] * inv) | (f8_pack2(v[2] * inv, v[3] * inv) << 16);
    q.y = f8_pack2(v[4] * inv, v[5] * inv) | (f8_pack2(v[6] * inv, v[7] * inv) << 16);
    const int nslot = p.pos ? p.k : 1;
    for (int i = 0; i < nslot; ++i) {
        const int64_t r = p.pos ? __ldcg(p.pos + row * p.k + i) : row;
        if (r < 0) continue;
        uint8_t* dst = p.q + r * p.cols + c0;
        if constexpr (VEC) {
            if (c0 < p.cols) *reinterpret_cast<uint2*>(dst) = q;
        } else {
#pragma unroll
            for (int b = 0; b < 8; ++b)
                if (c0 + b < p.cols)
                    dst[b] = static_cast<uint8_t>((b < 4 ? q.x : q.y) >> (8 * (b & 3)));
        }
        if (sub == 0) p.s[r * p.nblk + blk] = s;
    }
}

// ------------------------------------------------------------------- group
// Stable counting sort of the P = T k pairs by expert, in one CTA: warp w
// takes the w-th run of pairs, counts its experts, the counts are summed
// over (expert, warp), and a second pass over the run gives every pair its
// row.  Pairs whose expert lies outside [0, E) get row -1.
//   offsets[E+1]  first row of each expert, total last
//   pos[P]        row of each pair, or -1
constexpr int G_THREADS = 1024;
constexpr int G_WARPS = G_THREADS / 32;

__global__ void __launch_bounds__(G_THREADS) group_kernel(const int32_t* __restrict__ idx, int P,
                                                          int E, int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ pos) {
    extern __shared__ int hist[];  // [G_WARPS][E]
    __shared__ int wsum[G_WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < G_WARPS * E; i += G_THREADS) hist[i] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int run = ((P + G_WARPS - 1) / G_WARPS + 31) & ~31;
    const int beg = min(warp * run, P), end = min(beg + run, P);
    int* h = hist + warp * E;
    for (int i = beg; i < end; i += 32) {
        const int e = i + lane < end ? __ldcg(idx + i + lane) : -1;
        const bool in = e >= 0 && e < E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1);
        if (in && lane == __ffs(same) - 1) h[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // exclusive sums: over the warps of an expert, then over the experts
    int total = 0;
    if (tid < E)
        for (int w = 0; w < G_WARPS; ++w) {
            const int c = hist[w * E + tid];
            hist[w * E + tid] = total;
            total += c;
        }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    const int first = before + incl - total;
    if (tid < E) {
        offsets[tid] = first;
        if (tid == E - 1) offsets[E] = first + total;
        for (int w = 0; w < G_WARPS; ++w) hist[w * E + tid] += first;
    }
    __syncthreads();
    for (int i = beg; i < end; i += 32) {
        const int e = i + lane < end ? __ldcg(idx + i + lane) : -1;
        const bool in = e >= 0 && e < E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1);
        int row = -1;
        if (in) row = h[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (in && lane == __ffs(same) - 1) h[e] += __popc(same);
        __syncwarp();
        if (i + lane < end) pos[i + lane] = row;
    }
}

// ----------------------------------------------------------------- combine
// out[t] = residual[t] + sum_s w[t][s] y[pos[t][s]], summed in f32 in slot
// order and rounded once.  A thread takes four columns of one token.  Bound
// by reading y: 4 k bytes per output element.
constexpr int C_THREADS = 128;

template <class T>
__global__ void __launch_bounds__(C_THREADS) combine_kernel(
    const float* __restrict__ y, const int32_t* __restrict__ pos, const float* __restrict__ w,
    const T* residual, T* out, int H, int k) {
    const int64_t t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int c = (blockIdx.y * C_THREADS + threadIdx.x) * 4; c < H;
         c += gridDim.y * C_THREADS * 4) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < k; ++s) {
            const int r = __ldcg(pos + t * k + s);
            if (r < 0) continue;
            const float ws = __ldcg(w + t * k + s);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(r) * H + c));
            a[0] = fmaf(ws, v.x, a[0]);
            a[1] = fmaf(ws, v.y, a[1]);
            a[2] = fmaf(ws, v.z, a[2]);
            a[3] = fmaf(ws, v.w, a[3]);
        }
        const int64_t o = t * H + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = (residual ? to_f32(residual[o + i]) : 0.f) + a[i];
            if constexpr (sizeof(T) == 4) out[o + i] = v;
            else if constexpr (std::is_same<T, __half>::value) out[o + i] = __float2half_rn(v);
            else out[o + i] = __float2bfloat16_rn(v);
        }
    }
}

}  // namespace f8
}  // namespace qmoe
