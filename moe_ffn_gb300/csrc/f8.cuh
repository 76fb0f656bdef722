// f8.cuh — e4m3 values with one power-of-two scale per 128 of them.
//
// The scale of a block is the smallest s = 2^k, k >= -126, with
// max|x| <= 448 s (448 is the largest e4m3 value).  A power of two, because
// x / s is then exact and e4m3's own exponent loses nothing by it: a normal
// code keeps the same four significant bits whatever the power; only values
// below 2^-6 s (the subnormal codes; the block's largest exceeds 224 s unless k
// is -126, so at most 2^-13.8 of it) are coarser than with s = max|x| / 448, by
// at most one bit.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace qmoe {

constexpr int F8_BLOCK = 128;  // elements per scale along a row

// Bits of |v| where v is finite, else 0: the maximum over a block as an
// unsigned integer is its largest finite magnitude.
__device__ __forceinline__ uint32_t finite_abs_bits(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? b : 0u;
}

// Scale and its reciprocal (both exact powers of two) from the bits of the
// block's largest finite magnitude m 2^e, 1 <= m < 2: k = e - 8 if
// m <= 1.75, else e - 7 (448 = 1.75 * 2^8).  1 for a block of zeros.
__device__ __forceinline__ void f8_scale(uint32_t amax_bits, float* s, float* inv) {
    int k = static_cast<int>(amax_bits >> 23) - 127 - 8 +
            ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    k = max(k, -126);
    if (amax_bits == 0u) k = 0;
    *s = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    *inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
}

// Two values to e4m3, round to nearest even: `lo` in the low byte.  For values
// without infinities (the conversion saturates them).
__device__ __forceinline__ uint32_t f8_pack2_finite(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The same for any values: infinities become NaN, the only non-finite code.
__device__ __forceinline__ uint32_t f8_pack2(float lo, float hi) {
    lo = isinf(lo) ? __int_as_float(0x7FC00000) : lo;
    hi = isinf(hi) ? __int_as_float(0x7FC00000) : hi;
    return f8_pack2_finite(lo, hi);
}

}  // namespace qmoe
