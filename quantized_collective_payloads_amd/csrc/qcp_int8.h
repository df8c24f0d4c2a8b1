// qcp_int8.h -- a row's values to INT8 codes, as the quantize and the layer for few rows do it.
#pragma once

#include "qcp_device.h"

namespace qcp {

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));       // at an element's alignment

template <int T> constexpr int unit() { return T == F32 ? 4 : 8; }   // values of a piece

// a piece of x from p, of which `count` values exist (the others are zero)
template <int XT>
__device__ __forceinline__ u32x4_t load_piece(const void *p, int count) {
    if (count >= unit<XT>()) return __builtin_nontemporal_load((const u32x4_any *)p);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (XT == F32) {
            w[k] = k < count ? ((const uint32_t *)p)[k] : 0;
        } else {
            const uint16_t *h = (const uint16_t *)p;
            const uint32_t lo = 2 * k < count ? h[2 * k] : 0, hi = 2 * k + 1 < count ? h[2 * k + 1] : 0;
            w[k] = lo | (hi << 16);
        }
    }
    return u32x4_t{w[0], w[1], w[2], w[3]};
}

// the largest |x| of a piece and of m, on bit patterns: a NaN's is above infinity's.  Of
// 16-bit types m holds two maxima.
template <int XT>
__device__ __forceinline__ uint32_t largest(uint32_t m, u32x4_t v) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (XT == F32) {
            m = max(m, v[k] & 0x7fffffffu);
        } else {
            const u16x2_t a = __builtin_bit_cast(u16x2_t, m), b = __builtin_bit_cast(u16x2_t, v[k] & 0x7fff7fffu);
            m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
        }
    }
    return m;
}
// its fp32 bits
template <int XT>
__device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) {
    if constexpr (XT == F32) return m;
    m = max(m & 0xffffu, m >> 16);
    return XT == BF16 ? m << 16 : __float_as_uint(f16_lo(m));
}

// a piece -> its codes
template <int XT>
__device__ __forceinline__ u32x2_t encode(u32x4_t v, const BlockScale<INT8> &b, RecipBracket rb) {
    constexpr int U = unit<XT>();
    float x[U];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        if constexpr (XT == F32) {
            x[k] = __uint_as_float(v[k]);
        } else {
            x[2 * k] = widen_lo<XT>(v[k]);
            x[2 * k + 1] = widen_hi<XT>(v[k]);
        }
    }
    uint32_t t[U], diff = 0;
    if (b.fast) {
#pragma unroll
        for (int k = 0; k < U; k++) t[k] = int_code_bits_bracket(x[k], rb, diff);
        if (diff) {
#pragma unroll
            for (int k = 0; k < U; k++) t[k] = int_code_bits<INT8, true>(x[k], b);
        }
    } else {
#pragma unroll
        for (int k = 0; k < U; k++) t[k] = int_code_bits<INT8, false>(x[k], b);
    }
    u32x2_t c = {gather_low_bytes(t[0], t[1], t[2], t[3]), 0};
    if constexpr (XT != F32) c.y = gather_low_bytes(t[4], t[5], t[6], t[7]);
    return c;
}

// the scale of a row whose largest |x| has these fp32 bits; NaN where they are infinity's or a NaN's
__device__ __forceinline__ bool row_scale(uint32_t m, BlockScale<INT8> &b) {
    const bool finite = m < 0x7f800000u;
    b = block_scale<INT8>(finite ? __uint_as_float(m) : 0.0f);
    return finite;
}
__device__ __forceinline__ float scale_value(bool finite, const BlockScale<INT8> &b) {
    return finite ? b.s : __uint_as_float(0x7fc00000u);
}

}  // namespace qcp
