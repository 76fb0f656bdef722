// f8moe.cuh — the kernels around the e4m3 products: quantising rows, sorting
// a layer's (token, slot) pairs by expert, and adding the experts' outputs.
//
// Under programmatic dependent launch these grids may be resident while their
// inputs are still being written, so inputs are never read as data that is
// constant for the kernel's life (ld.global.nc): __ldcg, behind the wait.
#pragma once
#include "f8.cuh"
#include "gmm.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace qmoe {
namespace f8 {

// ---------------------------------------------------------------- quantise
// Sixteen lanes share a 128-column block, eight consecutive columns each:
// one or two 16-byte loads, a four-step maximum, one 8-byte store.  They take
// RUN neighbouring blocks of a row, all loaded before the first is reduced.
// Bound by HBM, (size + 1) bytes per element: RUN = 4 keeps 64 bytes per thread
// in flight (4096 x 14336 bf16: 29 us, 6.2 TB/s; with RUN = 1 42 us); RUN = 1
// spreads few rows over more threads (1 x 2048: 1.7 against 2.6 us).  VEC needs 16-byte aligned
// rows and whole groups of eight columns; the other form loads element by
// element.
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
    int nrun;         // runs of RUN blocks per row
};
constexpr int Q_THREADS = 256;

// Quantises a block held by sixteen lanes, eight values each: this lane's codes
// and the block's scale.  By a whole warp.
template <class T>
__device__ __forceinline__ uint2 quantize8(const Raw8<T>& x, float* scale) {
    uint32_t m = x.amax();
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    uint2 q;
    if (!__any_sync(0xffffffffu, m >= Raw8<T>::inf())) {
        f8_scale(Raw8<T>::f32_bits(m), scale, &inv);
        q.x = f8_pack2_finite(x.get(0) * inv, x.get(1) * inv) |
              (f8_pack2_finite(x.get(2) * inv, x.get(3) * inv) << 16);
        q.y = f8_pack2_finite(x.get(4) * inv, x.get(5) * inv) |
              (f8_pack2_finite(x.get(6) * inv, x.get(7) * inv) << 16);
        return q;
    }
    // infinities or NaN among the warp's values: the scale is the finite ones'
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, finite_abs_bits(x.get(i)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    f8_scale(m, scale, &inv);
    q.x = f8_pack2(x.get(0) * inv, x.get(1) * inv) |
          (f8_pack2(x.get(2) * inv, x.get(3) * inv) << 16);
    q.y = f8_pack2(x.get(4) * inv, x.get(5) * inv) |
          (f8_pack2(x.get(6) * inv, x.get(7) * inv) << 16);
    return q;
}

template <class T, bool VEC, int RUN>
__global__ void __launch_bounds__(Q_THREADS) quantize_kernel(const QuantParams p) {
    pdl_wait();
    pdl_trigger();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (Q_THREADS / 16) + (threadIdx.x >> 4);
    const int sub = threadIdx.x & 15;
    int64_t row;
    int blk0;
    if (p.rows * p.nrun <= 0x7fffffff) {
        row = static_cast<uint32_t>(item) / static_cast<uint32_t>(p.nrun);
        blk0 = (static_cast<int>(item) - static_cast<int>(row) * p.nrun) * RUN;
    } else {
        row = item / p.nrun;
        blk0 = static_cast<int>(item - row * p.nrun) * RUN;
    }
    const bool live = row < p.rows;
    const int nb = live ? min(RUN, p.nblk - blk0) : 0;
    const int c0 = blk0 * F8_BLOCK + sub * 8;
    const T* src = static_cast<const T*>(p.x) + (live ? row : 0) * p.ldx + c0;
    Raw8<T> v[RUN];
#pragma unroll
    for (int b = 0; b < RUN; ++b) {
        const int c = c0 + b * F8_BLOCK;
        v[b].zero();
        if (b < nb) {
            if constexpr (VEC) {
                if (c < p.cols) v[b].load(src + b * F8_BLOCK);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < p.cols)
                        reinterpret_cast<T*>(v[b].w)[i] = src[b * F8_BLOCK + i];
            }
        }
    }
    // the rows of a token's slots: one load, a slot per lane (k <= 16)
    const unsigned half = 0xffffu << (threadIdx.x & 16);
    const int slot_row = p.pos && live && sub < p.k ? __ldcg(p.pos + row * p.k + sub) : -1;
#pragma unroll
    for (int b = 0; b < RUN; ++b) {
        float s;
        const uint2 q = quantize8(v[b], &s);
        if (b >= nb) continue;
        const int c = c0 + b * F8_BLOCK;
        const int nslot = p.pos ? p.k : 1;
        for (int i = 0; i < nslot; ++i) {
            const int64_t r = p.pos ? __shfl_sync(half, slot_row, i, 16) : row;
            if (r < 0) continue;
            uint8_t* dst = p.q + r * p.cols + c;
            if constexpr (VEC) {
                if (c < p.cols) *reinterpret_cast<uint2*>(dst) = q;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c + e < p.cols)
                        dst[e] = static_cast<uint8_t>((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
            }
            if (sub == 0) p.s[r * p.nblk + blk0 + b] = s;
        }
    }
}

// ------------------------------------------------------------------- group
// Stable counting sort of the P = T k pairs by expert, in one cluster of up
// to eight CTAs.  Every warp takes one run of pairs and counts its experts;
// the counts are summed over (expert, CTA, warp), the CTAs' totals read from
// each other's shared memory, and a second pass over the run gives every pair
// its row.  Pairs whose expert lies outside [0, E) get row -1.  Bound by
// latency: G_AHEAD loads of a run are in flight at a time (32,768 pairs in 14 us;
// one CTA with one load in flight took 59).
//   offsets[E+1]  first row of each expert, total last
//   pos[P]        row of each pair, or -1
constexpr int G_THREADS = 1024;
constexpr int G_WARPS = G_THREADS / 32;
constexpr int G_AHEAD = 4;
constexpr int G_CLUSTER = 8;

__global__ void __launch_bounds__(G_THREADS) group_kernel(const int32_t* idx, int P, int E,
                                                          int32_t* offsets, int32_t* pos) {
    extern __shared__ int hist[];  // [G_WARPS][E], then this CTA's totals [E]
    __shared__ int wsum[G_WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    int* totals = hist + G_WARPS * E;
    for (int i = tid; i < G_WARPS * E; i += G_THREADS) hist[i] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int run = ((P + G_WARPS * ranks - 1) / (G_WARPS * ranks) + 31) & ~31;
    const int beg = min((rank * G_WARPS + warp) * run, P), end = min(beg + run, P);
    int* h = hist + warp * E;
    auto load = [&](int i, int (&e)[G_AHEAD]) {
#pragma unroll
        for (int a = 0; a < G_AHEAD; ++a) {
            const int j = i + 32 * a + lane;
            const int v = j < end ? __ldcg(idx + j) : -1;
            e[a] = v >= 0 && v < E ? v : -1;
        }
    };
    for (int i = beg; i < end; i += 32 * G_AHEAD) {
        int e[G_AHEAD];
        load(i, e);
#pragma unroll
        for (int a = 0; a < G_AHEAD; ++a) {
            if (i + 32 * a >= end) break;
            const unsigned same = __match_any_sync(0xffffffffu, e[a]);
            if (e[a] >= 0 && lane == __ffs(same) - 1) h[e[a]] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    // exclusive sums: over the warps of an expert, the CTAs, then the experts
    int mine = 0;
    if (tid < E) {
        for (int w = 0; w < G_WARPS; ++w) {
            const int c = hist[w * E + tid];
            hist[w * E + tid] = mine;
            mine += c;
        }
        totals[tid] = mine;
    }
    cluster_sync();
    int total = 0, before = 0;
    if (tid < E)
        for (int r = 0; r < ranks; ++r) {
            const int c = cluster_ld_s32(totals + tid, static_cast<uint32_t>(r));
            if (r < rank) before += c;
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
    int first = incl - total;
    for (int w = 0; w < warp; ++w) first += wsum[w];
    if (tid < E) {
        if (rank == 0) {
            offsets[tid] = first;
            if (tid == E - 1) offsets[E] = first + total;
        }
        for (int w = 0; w < G_WARPS; ++w) hist[w * E + tid] += first + before;
    }
    __syncthreads();
    for (int i = beg; i < end; i += 32 * G_AHEAD) {
        int e[G_AHEAD];
        load(i, e);
#pragma unroll
        for (int a = 0; a < G_AHEAD; ++a) {
            if (i + 32 * a >= end) break;
            const unsigned same = __match_any_sync(0xffffffffu, e[a]);
            int row = -1;
            if (e[a] >= 0) row = h[e[a]] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (e[a] >= 0 && lane == __ffs(same) - 1) h[e[a]] += __popc(same);
            __syncwarp();
            if (i + 32 * a + lane < end) pos[i + 32 * a + lane] = row;
        }
    }
    cluster_sync();  // no CTA leaves while another may read its totals
}

// ------------------------------------------------------- group + quantise
// Both steps for few pairs (P <= GQ_PAIRS), one CTA per token: every CTA reads
// all the expert indices and counts, for each of its token's slots, the pairs
// that come before it (smaller expert, or the same expert earlier); the first
// also counts the offsets.  One launch instead of two, whose cost is latency.
constexpr int GQ_PAIRS = 256;

template <class T>
__global__ void __launch_bounds__(Q_THREADS) group_quantize_kernel(
    const QuantParams p, const int32_t* idx, int P, int E, int32_t* offsets, int32_t* pos_out) {
    __shared__ int s_idx[GQ_PAIRS];
    __shared__ int s_pos[32];
    const int tid = threadIdx.x, t = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    for (int i = tid; i < P; i += Q_THREADS) {
        const int e = __ldcg(idx + i);
        s_idx[i] = e >= 0 && e < E ? e : -1;
    }
    if (tid < 32) s_pos[tid] = 0;
    __syncthreads();
    // a warp per slot
    for (int s = tid >> 5; s < p.k; s += Q_THREADS / 32) {
        const int me = t * p.k + s, e = s_idx[me];
        int n = 0;
        for (int i = tid & 31; i < P; i += 32) {
            const int o = s_idx[i];
            n += o >= 0 && (o < e || (o == e && i < me));
        }
        n = __reduce_add_sync(0xffffffffu, n);
        if ((tid & 31) == 0) {
            s_pos[s] = e < 0 ? -1 : n;
            pos_out[me] = e < 0 ? -1 : n;
        }
    }
    if (t == 0)
        for (int e = tid; e <= E; e += Q_THREADS) {
            int n = 0;
            for (int i = 0; i < P; ++i) n += s_idx[i] >= 0 && s_idx[i] < e;
            offsets[e] = n;
        }
    __syncthreads();
    const T* src = static_cast<const T*>(p.x) + t * p.ldx;
    const int sub = tid & 15;
    for (int b0 = 0; b0 < p.nblk; b0 += Q_THREADS / 16) {
        const int b = b0 + (tid >> 4);
        const int c = b * F8_BLOCK + sub * 8;
        Raw8<T> v;
        v.zero();
        if (b < p.nblk) v.load(src + c);
        float s;
        const uint2 q = quantize8(v, &s);
        if (b >= p.nblk) continue;
        for (int i = 0; i < p.k; ++i) {
            const int64_t r = s_pos[i];
            if (r < 0) continue;
            *reinterpret_cast<uint2*>(p.q + r * p.cols + c) = q;
            if (sub == 0) p.s[r * p.nblk + b] = s;
        }
    }
}

// ----------------------------------------------------------------- combine
// out[t] = residual[t] + sum_s w[t][s] y[pos[t][s]], summed in f32 in slot
// order and rounded once.  A thread takes eight columns of one token and eight
// slots at a step (1 / 512 / 4096 tokens of top-8, cold: 5.7 / 7.4 / 28 us; four at
// a step 6.3 / 7.9 / 29; rows and weights of the slots loaded by every thread
// instead of once per warp 7.6 / 9.2 / 39).  Bound by reading y: for bf16
// activations y is bf16 (the layer rounds each expert's output once, by at most
// 2^-8 of it, as out's own rounding is of out; y is the layer's largest traffic),
// else f32.  Both sides for bf16 activations, 4096 tokens, hidden 2048, 128
// experts, top-8, F 768: y in bf16 364 us and 1.77e-3 root mean square error
// against 64 bits, in f32 459 us and 1.66e-3 (the rounding of out alone); 512
// tokens, 64 experts, F 1024: 109 us and 1.80e-3 against 125 and 1.66e-3.  A
// caller who wants f32 sums throughout passes f32 activations.
constexpr int C_THREADS = 128;
constexpr int C_AHEAD = 8;

template <class T, class Y>
__global__ void __launch_bounds__(C_THREADS) combine_kernel(
    const Y* y, const int32_t* pos, const float* w, const T* residual, T* out, int H, int k) {
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * C_THREADS + threadIdx.x) * 8;
    const int lane = threadIdx.x & 31;
    const bool in = c < H;
    pdl_wait();
    pdl_trigger();
    // a token's slots: one load, a slot per lane (k <= 16)
    const int slot_row = lane < k ? __ldcg(pos + t * k + lane) : -1;
    const float slot_w = lane < k ? __ldcg(w + t * k + lane) : 0.f;
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = 0.f;
    for (int s0 = 0; s0 < k; s0 += C_AHEAD) {
        Raw8<Y> v[C_AHEAD];
        float ws[C_AHEAD];
        int r[C_AHEAD];
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s) {
            r[s] = __shfl_sync(0xffffffffu, slot_row, s0 + s);  // -1 past the slots
            ws[s] = __shfl_sync(0xffffffffu, slot_w, s0 + s);
            if (r[s] < 0) ws[s] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s) {
            v[s].zero();
            if (in && r[s] >= 0) v[s].load(y + static_cast<int64_t>(r[s]) * H + c);
        }
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = fmaf(ws[s], v[s].get(i), a[i]);
    }
    if (!in) return;
    if (residual) {
        float r[8];
        load8(residual + t * H + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] += r[i];
    }
    store8(out + t * H + c, a);
}

}  // namespace f8
}  // namespace qmoe
