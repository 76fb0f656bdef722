// moe_steps.cuh — the steps of a mixture-of-experts layer around its experts'
// products: routing, the sort of the tokens by expert, and the weighted sum of the
// experts' outputs, each with its gradient.
//
// Under programmatic dependent launch these grids may be resident while their
// inputs are still being written: every load of them lies behind the wait and goes
// through __ldcg.
#pragma once
#include "ptx.cuh"
#include "route.cuh"
#include "rows.cuh"

namespace qmoe {
namespace steps {

constexpr int MAX_EXPERTS = 1024;
constexpr int MAX_TOPK = 16;  // a token's slots lie in the lanes of one warp

// ------------------------------------------------------------------ routing
// A warp per token; lane i holds the logits i V .. i V + V - 1.  Each lane sorts its own
// once, best first, and each of the k rounds takes the best of the lanes' heads, so that a
// round costs one warp maximum and a shift of one lane's list.  16-bit logits rank by one
// 32-bit word, the ranking key of route.cuh's rule above the inverted index, whose
// maximum is the winner, index and all; f32 logits need the key's 32 bits for themselves,
// and the lowest lane with the largest key then has the lowest index among equals.
// Bound by launch for few tokens (1 x 128: 1.7 us), by instruction issue for many (16,384 x
// 128 bf16, top-8: 6.9 us of 0.8 for the bytes, not renormalised 7.7; issue 75%, ALU 63%;
// the gradient 6.4, not renormalised 7.2).  Both together, not renormalised, 14.3; with a
// maximum over all V values in each round and the gradient's slots searched 18.8.  256 / 512 /
// 1024 experts: 10.2 / 19.2 / 73 us (from V = 32 on, f32 from 16, the compiler does not unroll
// the network, and the lists lie in local memory).
constexpr int R_WARPS = 4;

struct RouteParams {
    const void* logits;
    int64_t ldl;
    int64_t n_tokens;
    int E, k;
    bool vec;       // whole aligned runs of V logits
    bool renorm;
    int32_t* idx;
    float* w;
    // backward
    const float* grad_w;
    void* grad;     // logits' type
    int64_t ldg;
    bool vec_g;
};

// V values of a row from element c on, as f32; `fill` past the row's end.
template <class T, int V>
__device__ __forceinline__ void load_run(const T* row, int c, int E, bool vec, float fill,
                                         float (&v)[V]) {
    constexpr int BYTES = V * static_cast<int>(sizeof(T));
    if constexpr (BYTES >= 4) {
        if (vec) {  // E is a multiple of V: a lane's run is whole or empty
            uint32_t w[BYTES / 4];
            if (c < E) {
                const T* p = row + c;
                if constexpr (BYTES >= 16) {
#pragma unroll
                    for (int i = 0; i < BYTES / 16; ++i) {
                        const uint4 a = __ldcg(reinterpret_cast<const uint4*>(p) + i);
                        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
                    }
                } else if constexpr (BYTES == 8) {
                    const uint2 a = __ldcg(reinterpret_cast<const uint2*>(p));
                    w[0] = a.x; w[1] = a.y;
                } else {
                    w[0] = __ldcg(reinterpret_cast<const uint32_t*>(p));
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
                    else v[i] = to_f32(reinterpret_cast<const T*>(w)[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = fill;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = c + i < E ? to_f32(ldcg_value(row + c + i)) : fill;
}

// A sorting network (Batcher's odd-even merge sort) over V items held in registers, larger
// first.
template <int V, class Swap>
__device__ __forceinline__ void sort_network(Swap swap) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p))
                        swap(i + j, i + j + k);
}

// Ranking key of a 16-bit logit's bits by route.cuh's rule, as 16 bits, and the value of
// a key.
template <class T>
__device__ __forceinline__ uint32_t key16(uint32_t b) {
    constexpr uint32_t inf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    if ((b & 0x7FFFu) > inf) return 0xFFFFu;   // NaN
    if ((b & 0x7FFFu) == 0u) b = 0u;           // -0 ranks as +0
    return (b & 0x8000u) ? ~b & 0xFFFFu : b | 0x8000u;
}
template <class T>
__device__ __forceinline__ float key16_value(uint32_t k) {
    const unsigned short b =
        static_cast<unsigned short>((k & 0x8000u) ? k & 0x7FFFu : ~k & 0xFFFFu);
    return to_f32(*reinterpret_cast<const T*>(&b));
}

__device__ __forceinline__ float warp_sum(float z) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    return z;
}

// The k best of a warp's logits: lane s gets the s-th's index and value; all lanes the
// best value.
template <class T, int V>
__device__ __forceinline__ float take_best(const float (&v)[V], int c, int E, int k, int lane,
                                           int* idx, float* value) {
    if constexpr (sizeof(T) == 2) {
        uint32_t w[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const T raw = from_f32<T>(v[i]);  // (exact: it came from there)
            const uint32_t b = *reinterpret_cast<const unsigned short*>(&raw);
            w[i] = c + i < E ? key16<T>(b) << 16 | (0xFFFFu - (c + i)) : 0u;
        }
        sort_network<V>([&](int i, int j) {
            const uint32_t hi = max(w[i], w[j]), lo = min(w[i], w[j]);
            w[i] = hi;
            w[j] = lo;
        });
        uint32_t mine = 0, top = 0;
        for (int s = 0; s < k; ++s) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, w[0]);
            if (s == 0) top = m;
            if (lane == s) mine = m;
            const bool won = w[0] == m;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t next = i + 1 < V ? w[i + 1] : 0u;
                w[i] = won ? next : w[i];
            }
        }
        *idx = static_cast<int>(0xFFFFu - (mine & 0xFFFFu));
        *value = key16_value<T>(mine >> 16);
        return key16_value<T>(top >> 16);
    } else {
        uint32_t key[V];  // 0: none left (no key is 0)
        int at[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = c + i < E ? route_key(v[i]) : 0u;
            at[i] = c + i;
        }
        sort_network<V>([&](int i, int j) {
            const bool ok = key[i] > key[j] || (key[i] == key[j] && at[i] < at[j]);
            const uint32_t hi = ok ? key[i] : key[j], lo = ok ? key[j] : key[i];
            const int first = ok ? at[i] : at[j], second = ok ? at[j] : at[i];
            key[i] = hi;
            key[j] = lo;
            at[i] = first;
            at[j] = second;
        });
        uint32_t mine = 0, top = 0;
        int index = 0;
        for (int s = 0; s < k; ++s) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
            const int who = __ffs(__ballot_sync(0xffffffffu, key[0] == m)) - 1;
            const int e = __shfl_sync(0xffffffffu, at[0], who);
            if (s == 0) top = m;
            if (lane == s) {
                mine = m;
                index = e;
            }
            const bool won = lane == who;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t next = i + 1 < V ? key[i + 1] : 0u;
                key[i] = won ? next : key[i];
                if (i + 1 < V) at[i] = won ? at[i + 1] : at[i];
            }
        }
        *idx = index;
        *value = route_key_value(mine);
        return route_key_value(top);
    }
}

template <class T, int V>
__global__ void __launch_bounds__(R_WARPS * 32) route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * R_WARPS + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (t >= p.n_tokens) return;
    const int c = lane * V;
    float v[V];
    load_run<T, V>(static_cast<const T*>(p.logits) + t * p.ldl, c, p.E, p.vec, 0.f, v);
    int idx;
    float value;
    const float top = take_best<T, V>(v, c, p.E, p.k, lane, &idx, &value);
    float w;
    if (route_degenerate(top)) {
        idx = lane;
        w = __int_as_float(0x7FC00000);
    } else {
        const float x = lane < p.k ? expf(value - top) : 0.f;
        float z = x;
        if (!p.renorm) {
            z = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < p.E) z += expf(v[i] - top);
        }
        w = x / warp_sum(z);
    }
    if (lane < p.k) {
        p.idx[t * p.k + lane] = idx;
        p.w[t * p.k + lane] = w;
    }
}

// Gradient of the logits, a warp per token, with c = sum_s w_s dw_s over the slots
// that name an expert:
//   renormalised      dl_e = sum over slots s of e: w_s (dw_s - c)
//   not renormalised  dl_e = p_e ((sum over slots s of e: dw_s) - c), p the softmax
//                     over all experts, formed again from the logits
// The slots' terms are scattered through shared memory; where two slots of a token name
// one expert, which moe_route never does, they are added in slot order.
template <class T, int V>
__global__ void __launch_bounds__(R_WARPS * 32) route_backward_kernel(const RouteParams p) {
    __shared__ float s_row[R_WARPS][32 * V];
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * R_WARPS + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (t >= p.n_tokens) return;
    const int c = lane * V;
    float* row = s_row[threadIdx.x >> 5];
    int idx = lane < p.k ? __ldcg(p.idx + t * p.k + lane) : -1;
    const bool live = idx >= 0 && idx < p.E;
    if (!live) idx = -1 - lane;  // (distinct)
    const float w = live ? __ldcg(p.w + t * p.k + lane) : 0.f;
    const float d = live ? __ldcg(p.grad_w + t * p.k + lane) : 0.f;
    float v[V], g[V];
    if (!p.renorm)
        load_run<T, V>(static_cast<const T*>(p.logits) + t * p.ldl, c, p.E, p.vec,
                       -__int_as_float(0x7F800000), v);
#pragma unroll
    for (int i = 0; i < V; ++i) row[c + i] = 0.f;
    const float dot = warp_sum(w * d);
    const float mine = p.renorm ? w * (d - dot) : d;
    const unsigned same = __match_any_sync(0xffffffffu, idx);
    __syncwarp();
    if (!__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        if (live) row[idx] = mine;
    } else {
        for (int s = 0; s < p.k; ++s) {
            if (lane == s && live) row[idx] += mine;
            __syncwarp();
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = row[c + i];
    if (!p.renorm) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, c + i < p.E ? route_key(v[i]) : 0u);
        const float top = route_key_value(__reduce_max_sync(0xffffffffu, best));
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = c + i < p.E ? expf(v[i] - top) : 0.f;
            z += v[i];
        }
        const float inv = 1.f / warp_sum(z);
#pragma unroll
        for (int i = 0; i < V; ++i)
            g[i] = route_degenerate(top) ? __int_as_float(0x7FC00000) : v[i] * inv * (g[i] - dot);
    }
    T* out = static_cast<T*>(p.grad) + t * p.ldg + c;
    constexpr int BYTES = V * static_cast<int>(sizeof(T));
    if constexpr (BYTES >= 4) {
        if (p.vec_g) {
            if (c >= p.E) return;
            uint32_t q[BYTES / 4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (sizeof(T) == 4) q[i] = __float_as_uint(g[i]);
                else reinterpret_cast<T*>(q)[i] = from_f32<T>(g[i]);
            }
            if constexpr (BYTES >= 16) {
#pragma unroll
                for (int i = 0; i < BYTES / 16; ++i)
                    reinterpret_cast<uint4*>(out)[i] =
                        make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
            } else if constexpr (BYTES == 8) {
                *reinterpret_cast<uint2*>(out) = make_uint2(q[0], q[1]);
            } else {
                *reinterpret_cast<uint32_t*>(out) = q[0];
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < p.E) out[i] = from_f32<T>(g[i]);
}

// ------------------------------------------------------------------ permute
// Stable counting sort of the P = T k (token, slot) pairs by expert, and the copy
// of each token's row to its pairs' rows, read once and written k times.
//
// A CTA takes a run of tokens.  A pair's row is the number of pairs of smaller
// experts, plus the pairs of its expert in earlier runs, plus those before it in
// its own run.  The first two come from all the indices, counted by every CTA
// for itself, while they are few (up to P_ALONE pairs: one launch), else from a
// table of counts [runs][Ep] that count_kernel makes, eight experts to a load.
// The rows to copy do not depend on any of it: they are on their way to registers
// (four segments of a row per warp) while their places are found.
// Bound by writing the rows: 4096 x 2048 bf16, top-8, 128 experts 27.4 us (5.5 TB/s; the
// counts 2 us of it, finding the places about 3).  Called in turn 28.2; with the rows loaded
// after their places were known and two bytes of counts to a load 44.6.  1 x 2048: 3.2 us, latency.
constexpr int P_THREADS = 256;
constexpr int P_WARPS = P_THREADS / 32;
constexpr int P_ALONE = 8192;
constexpr int P_POS = 1024;   // positions of a run kept in shared memory
constexpr int P_AHEAD = 4;    // units of a lane in a segment of a row
constexpr int P_EARLY = 4;    // segments loaded before their places are known

struct PermuteParams {
    const uint8_t* x;
    int64_t ldx;            // bytes
    uint8_t* rows;
    int64_t ldr;            // bytes
    int nvec;               // units of VB bytes in a row
    const int32_t* idx;
    int32_t* offsets;
    int32_t* pos;
    int P, E, k;
    int Ep;                 // experts, rounded up to eight
    int run;                // tokens of a run
    int runs;
    uint16_t* counts;       // [runs][Ep], or null
};

// The expert of pair i, or -1.
__device__ __forceinline__ int expert_of(const int32_t* idx, int i, int E) {
    const int e = __ldcg(idx + i);
    return e >= 0 && e < E ? e : -1;
}

__global__ void __launch_bounds__(P_THREADS) count_kernel(const PermuteParams p) {
    extern __shared__ int hist[];
    const int tid = threadIdx.x;
    for (int e = tid; e < p.Ep; e += P_THREADS) hist[e] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int beg = blockIdx.x * p.run * p.k, end = min(beg + p.run * p.k, p.P);
    for (int i = beg + tid; i < end; i += P_THREADS) {
        const int e = expert_of(p.idx, i, p.E);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    uint16_t* out = p.counts + static_cast<int64_t>(blockIdx.x) * p.Ep;
    for (int e = tid; e < p.Ep; e += P_THREADS) out[e] = static_cast<uint16_t>(hist[e]);
}

template <int VB>
struct Unit;
template <> struct Unit<16> { using type = uint4; };
template <> struct Unit<4> { using type = uint32_t; };
template <> struct Unit<2> { using type = uint16_t; };

// STREAM: rows that L2 does not hold, written evict-first.
template <int VB, bool STREAM>
__global__ void __launch_bounds__(P_THREADS) permute_kernel(const PermuteParams p) {
    using U = typename Unit<VB>::type;
    extern __shared__ int sm[];
    __shared__ int s_pos[P_POS];
    __shared__ int s_wsum[P_WARPS];
    int* whist = sm;                    // [P_WARPS][Ep] this run's counts, then next rows
    int* total = sm + P_WARPS * p.Ep;   // [Ep]
    int* before = total + p.Ep;         // [Ep]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = blockIdx.x;
    for (int i = tid; i < (P_WARPS + 2) * p.Ep; i += P_THREADS) sm[i] = 0;
    pdl_wait();
    pdl_trigger();
    const int beg = r * p.run * p.k, end = min(beg + p.run * p.k, p.P);
    // (token, segment) items, spread over the warps of all CTAs of this run
    const int ntok = (end - beg) / p.k;
    const int nseg = (p.nvec + 32 * P_AHEAD - 1) / (32 * P_AHEAD);
    const int64_t items = static_cast<int64_t>(ntok) * nseg;
    const int64_t it0 = blockIdx.y * P_WARPS + warp, it_step = gridDim.y * P_WARPS;
    auto load = [&](int64_t it, U (&u)[P_AHEAD]) {
        if (it >= items) return;
        const int tok = static_cast<int>(it / nseg);
        const int v0 = static_cast<int>(it - static_cast<int64_t>(tok) * nseg) * 32 * P_AHEAD + lane;
        const U* src = reinterpret_cast<const U*>(p.x + (static_cast<int64_t>(r) * p.run + tok) *
                                                            p.ldx);
#pragma unroll
        for (int a = 0; a < P_AHEAD; ++a)
            if (v0 + 32 * a < p.nvec) u[a] = __ldcg(src + v0 + 32 * a);
    };
    auto store = [&](int64_t it, const U (&u)[P_AHEAD]) {
        if (it >= items) return;
        const int tok = static_cast<int>(it / nseg);
        const int v0 = static_cast<int>(it - static_cast<int64_t>(tok) * nseg) * 32 * P_AHEAD + lane;
        for (int s = 0; s < p.k; ++s) {
            const int i = tok * p.k + s;
            const int row = i < P_POS ? s_pos[i] : __ldcg(p.pos + beg + i);
            if (row < 0) continue;
            U* dst = reinterpret_cast<U*>(p.rows + static_cast<int64_t>(row) * p.ldr);
#pragma unroll
            for (int a = 0; a < P_AHEAD; ++a)
                if (v0 + 32 * a < p.nvec) {
                    if constexpr (STREAM) __stcs(dst + v0 + 32 * a, u[a]);
                    else dst[v0 + 32 * a] = u[a];
                }
        }
    };
    // this run's pairs, a part to each warp, the first 32 of it in registers
    const int part = ((end - beg + P_WARPS - 1) / P_WARPS + 31) & ~31;
    const int wbeg = min(beg + warp * part, end), wend = min(wbeg + part, end);
    const int head_idx = wbeg + lane < wend ? __ldcg(p.idx + wbeg + lane) : -1;
    U early[P_EARLY][P_AHEAD];
#pragma unroll
    for (int i = 0; i < P_EARLY; ++i) load(it0 + i * it_step, early[i]);
    __syncthreads();
    if (p.counts) {
        // eight experts to a thread, the runs spread over the groups of threads that
        // cover them all
        const int per = p.Ep / 8, groups = P_THREADS / per;
        const int group = tid / per, e0 = (tid - group * per) * 8;
        if (group < groups) {
            int all[8], ahead[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) all[i] = ahead[i] = 0;
#pragma unroll 8
            for (int j = group; j < p.runs; j += groups) {
                const uint4 q = __ldcg(reinterpret_cast<const uint4*>(
                    p.counts + static_cast<int64_t>(j) * p.Ep + e0));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = static_cast<int>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
                    all[i] += n;
                    ahead[i] += j < r ? n : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (all[i]) atomicAdd(&total[e0 + i], all[i]);
                if (ahead[i]) atomicAdd(&before[e0 + i], ahead[i]);
            }
        }
    } else {
        // (both counts in one word: there are at most 8192 pairs)
#pragma unroll 8
        for (int i = tid; i < p.P; i += P_THREADS) {
            const int e = expert_of(p.idx, i, p.E);
            if (e >= 0) atomicAdd(&total[e], i < beg ? 0x10001 : 0x10000);
        }
    }
    const int head = head_idx >= 0 && head_idx < p.E ? head_idx : -1;
    int* h = whist + warp * p.Ep;
    for (int i = wbeg; i < wend; i += 32) {
        const int e = i == wbeg ? head : i + lane < wend ? expert_of(p.idx, i + lane, p.E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) h[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // exclusive sum over the experts, a run of experts to each thread
    const int per = (p.E + P_THREADS - 1) / P_THREADS;
    const int e0 = min(tid * per, p.E), e1 = min(e0 + per, p.E);
    auto total_of = [&](int e) { return p.counts ? total[e] : total[e] >> 16; };
    int mine = 0;
    for (int e = e0; e < e1; ++e) mine += total_of(e);
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_wsum[warp] = incl;
    __syncthreads();
    int first = incl - mine;
    for (int w = 0; w < warp; ++w) first += s_wsum[w];
    const bool tell = r == 0 && blockIdx.y == 0;
    for (int e = e0; e < e1; ++e) {
        if (tell) p.offsets[e] = first;
        int at = first + (p.counts ? before[e] : total[e] & 0xFFFF);
        first += total_of(e);
#pragma unroll
        for (int w = 0; w < P_WARPS; ++w) {
            const int n = whist[w * p.Ep + e];
            whist[w * p.Ep + e] = at;
            at += n;
        }
        if (tell && e == p.E - 1) p.offsets[p.E] = first;
    }
    __syncthreads();
    for (int i = wbeg; i < wend; i += 32) {
        const int e = i == wbeg ? head : i + lane < wend ? expert_of(p.idx, i + lane, p.E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = h[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) h[e] += __popc(same);
        __syncwarp();
        if (i + lane < wend) {
            p.pos[i + lane] = row;  // (the same value from every blockIdx.y)
            if (i + lane - beg < P_POS) s_pos[i + lane - beg] = row;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P_EARLY; ++i) store(it0 + i * it_step, early[i]);
    for (int64_t it = it0 + P_EARLY * it_step; it < items; it += it_step) {
        U u[P_AHEAD];
        load(it, u);
        store(it, u);
    }
}

// ------------------------------------------------------------------ combine
// out[t] = residual[t] + sum_s w[t][s] y[pos[t][s]], summed in f32 in slot order and
// rounded once.  A thread takes N columns of one token (N = 8 where every row is
// whole aligned 16-byte units, else 1), eight slots at a step.  Bound by reading y: 4096 x
// 2048 bf16, top-8 27 us (6.2 TB/s) with inputs that L2 does not hold; single columns 517 x
// 2065 f32, top-6 6.2 us, where whole units take 7.1 for 2064.
constexpr int C_THREADS = 128;
constexpr int C_AHEAD = 8;
// Threads of the sum's CTAs: 64 take 512 columns of whole units (4096 x 2048 top-8: 28.3 us, 128
// threads 29.3, 256 30.1), 128 single columns (1000 x 1111: 10.5 us, 64 threads 19.0).
template <int N>
constexpr int SUM_THREADS = N == 8 ? 64 : 128;
// Groups of N columns a thread takes, a CTA's width apart.
template <int N>
constexpr int SUM_GROUPS = N == 8 ? 1 : 4;

struct CombineParams {
    const void* y;
    int64_t n_rows, ldy;
    int cols;
    const int32_t* pos;
    const float* w;         // null: ones
    int k;
    const void* residual;   // null: zeros
    void* out;
    int64_t ldo;
    // backward
    const void* grad_out;   // rows ldo apart
    void* grad_y;           // null: not wanted
    int64_t ldg;
    float* grad_w;          // null: not wanted
};

// Eight values that are not read again by this call: evicted first from L2, where other
// operands may still be wanted.
template <class T>
__device__ __forceinline__ void load_once(Raw8<T>& v, const T* p, uint64_t policy) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        asm volatile(
            "ld.relaxed.gpu.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
            : "=r"(v.w[4 * i]), "=r"(v.w[4 * i + 1]), "=r"(v.w[4 * i + 2]), "=r"(v.w[4 * i + 3])
            : "l"(reinterpret_cast<const uint4*>(p) + i), "l"(policy));
}
// One value, with the interface of Raw8.
template <class T>
struct Raw1 {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = ldcg_value(p); }
    __device__ __forceinline__ void zero() { v = from_f32<T>(0.f); }
    __device__ __forceinline__ float get(int) const { return to_f32(v); }
};
// N consecutive values of a row.
template <class T, int N>
using Run = typename std::conditional<N == 8, Raw8<T>, Raw1<T>>::type;
template <class T, int N>
__device__ __forceinline__ void store_run(T* p, const float (&v)[N]) {
    if constexpr (N == 8) store8(p, v);
    else p[0] = from_f32<T>(v[0]);
}

// A token's slots: one load, a slot per lane (k <= 16); a row outside [0, n_rows)
// adds nothing.
__device__ __forceinline__ void load_slots(const CombineParams& p, int64_t t, int lane, int* row,
                                           float* w) {
    int r = lane < p.k ? __ldcg(p.pos + t * p.k + lane) : -1;
    if (r >= p.n_rows) r = -1;
    *row = r;
    *w = r >= 0 ? (p.w ? __ldcg(p.w + t * p.k + lane) : 1.f) : 0.f;
}

template <class Y, class O, int N>
__global__ void __launch_bounds__(SUM_THREADS<N>) combine_kernel(const CombineParams p) {
    constexpr int G = SUM_GROUPS<N>, STEP = SUM_THREADS<N> * N;
    const int64_t t = blockIdx.x;
    const int c0 = blockIdx.y * G * STEP + threadIdx.x * N;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const uint64_t once = policy_evict_first();
    int slot_row;
    float slot_w;
    load_slots(p, t, lane, &slot_row, &slot_w);
    float a[G][N];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < N; ++i) a[g][i] = 0.f;
    for (int s0 = 0; s0 < p.k; s0 += C_AHEAD) {
        Run<Y, N> v[C_AHEAD][G];
        float w[C_AHEAD];
        int r[C_AHEAD];
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s) {
            r[s] = __shfl_sync(0xffffffffu, slot_row, s0 + s);  // -1 past the slots
            w[s] = __shfl_sync(0xffffffffu, slot_w, s0 + s);
        }
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s) {
            const Y* at = static_cast<const Y*>(p.y) + static_cast<int64_t>(r[s]) * p.ldy + c0;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                v[s][g].zero();
                if (r[s] < 0 || c0 + g * STEP >= p.cols) continue;
                if constexpr (N == 8) load_once(v[s][g], at + g * STEP, once);
                else v[s][g].load(at + g * STEP);
            }
        }
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s)
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) a[g][i] = fmaf(w[s], v[s][g].get(i), a[g][i]);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int c = c0 + g * STEP;
        if (c >= p.cols) continue;
        if (p.residual) {
            Run<O, N> q;
            q.load(static_cast<const O*>(p.residual) + t * p.ldo + c);
#pragma unroll
            for (int i = 0; i < N; ++i) a[g][i] += q.get(i);
        }
        store_run<O, N>(static_cast<O*>(p.out) + t * p.ldo + c, a[g]);
    }
}

// Gradients: of a row, grad_y[pos[t][s]] = w[t][s] grad_out[t], rounded once; of a
// weight, grad_w[t][s] = sum_c y[pos[t][s]][c] grad_out[t][c] in f32 (0 for a slot
// without a row).  A CTA per token reads grad_out and the token's rows once.  Bound by HBM:
// 4096 x 2048 bf16, top-8 46 us (285 MB, 6.2 TB/s).
template <class Y, class O, int N>
__global__ void __launch_bounds__(C_THREADS) combine_backward_kernel(const CombineParams p) {
    __shared__ float s_sum[C_THREADS / 32][MAX_TOPK];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    int slot_row;
    float slot_w;
    load_slots(p, t, lane, &slot_row, &slot_w);
    const O* g_row = static_cast<const O*>(p.grad_out) + t * p.ldo;
    for (int s0 = 0; s0 < p.k; s0 += C_AHEAD) {
        float w[C_AHEAD], sum[C_AHEAD];
        int r[C_AHEAD];
#pragma unroll
        for (int s = 0; s < C_AHEAD; ++s) {
            r[s] = __shfl_sync(0xffffffffu, slot_row, s0 + s);
            w[s] = __shfl_sync(0xffffffffu, slot_w, s0 + s);
            sum[s] = 0.f;
        }
        for (int c = tid * N; c < p.cols; c += C_THREADS * N) {
            Run<O, N> g;
            Run<Y, N> v[C_AHEAD];
            g.load(g_row + c);
            if (p.grad_w) {
#pragma unroll
                for (int s = 0; s < C_AHEAD; ++s) {
                    v[s].zero();
                    if (r[s] >= 0)
                        v[s].load(static_cast<const Y*>(p.y) + static_cast<int64_t>(r[s]) * p.ldy +
                                  c);
                }
#pragma unroll
                for (int s = 0; s < C_AHEAD; ++s)
                    if (r[s] >= 0)
#pragma unroll
                        for (int i = 0; i < N; ++i) sum[s] = fmaf(v[s].get(i), g.get(i), sum[s]);
            }
            if (p.grad_y) {
#pragma unroll
                for (int s = 0; s < C_AHEAD; ++s)
                    if (r[s] >= 0) {
                        float d[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) d[i] = w[s] * g.get(i);
                        store_run<Y, N>(static_cast<Y*>(p.grad_y) +
                                            static_cast<int64_t>(r[s]) * p.ldg + c, d);
                    }
            }
        }
        if (p.grad_w) {
#pragma unroll
            for (int s = 0; s < C_AHEAD; ++s) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    sum[s] += __shfl_xor_sync(0xffffffffu, sum[s], o);
                if (lane == 0) s_sum[tid >> 5][s0 + s] = sum[s];
            }
        }
    }
    if (!p.grad_w) return;
    __syncthreads();
    if (tid < p.k) {
        float a = 0.f;
        for (int i = 0; i < C_THREADS / 32; ++i) a += s_sum[i][tid];
        p.grad_w[t * p.k + tid] = a;
    }
}

}  // namespace steps
}  // namespace qmoe
