// rows.cuh — rows of f32, bf16 and f16 values: conversions, eight values at a
// time, and how they are loaded and stored.
//
// Loads go through __ldcg: a grid launched early (programmatic dependent launch)
// may be resident while its inputs are still being written, so nothing is read as
// data that is constant for the kernel's life.
#pragma once
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace qmoe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __float2bfloat16_rn(v);
    else return v;
}
// One value of any of the types.
template <class T>
__device__ __forceinline__ T ldcg_value(const T* p) {
    if constexpr (sizeof(T) == 4) {
        return __ldcg(p);
    } else {
        const unsigned short u = __ldcg(reinterpret_cast<const unsigned short*>(p));
        return *reinterpret_cast<const T*>(&u);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive values as they lie in memory.
template <class T>
struct Raw8 {
    uint32_t w[sizeof(T) * 2];
    __device__ __forceinline__ void load(const T* src) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
            const uint4 a = __ldcg(reinterpret_cast<const uint4*>(src) + i);
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)) * 2; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return to_f32(reinterpret_cast<const T*>(w)[i]);
    }
    // The largest magnitude as its type's bits (16-bit values two at a time):
    // magnitudes order as their bits do, infinities and NaN above the rest.
    __device__ __forceinline__ uint32_t amax() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        } else {
            uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
            return max(m & 0xFFFFu, m >> 16);
        }
    }
    static __device__ __forceinline__ uint32_t inf() {
        return sizeof(T) == 4 ? 0x7F800000u : std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
    }
    // f32 bits of a magnitude from its type's
    static __device__ __forceinline__ uint32_t f32_bits(uint32_t m) {
        if constexpr (sizeof(T) == 4)
            return m;
        else if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(
                __half2float(__ushort_as_half(static_cast<unsigned short>(m))));
        else
            return m << 16;
    }
};

template <class T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
    Raw8<T> r;
    r.load(src);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
}
template <class T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 q;
        uint32_t* u = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = std::is_same<T, __half>::value ? pack_f16(v[2 * i], v[2 * i + 1])
                                                  : pack_bf16(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4*>(dst) = q;
    }
}

}  // namespace qmoe
