// mq_mx4_device.hpp -- device helpers of the microscaled 4-bit linear layers (gfx950).
#pragma once

#include "mq_device.hpp"
#include "mq_mx4.hpp"

namespace mq {

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

// Element types of dense matrices.
template <int DT> struct Dense;
template <> struct Dense<MQ_BF16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(T b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ T store(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
};
template <> struct Dense<MQ_F16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(T b) { return (float)__builtin_bit_cast(_Float16, b); }
    static __device__ __forceinline__ T store(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
template <> struct Dense<MQ_F32> {
    typedef float T;
    static __device__ __forceinline__ float load(T v) { return v; }
    static __device__ __forceinline__ T store(float v) { return v; }
};

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`: the smallest power of
// two with amax <= 6 = 1.5 * 2^2 of it; 255 for a NaN or an infinity (their bits exceed every
// finite magnitude's).
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax)
{
    const int e = (int)(amax >> 23) - 2 + ((amax & 0x7FFFFFu) > 0x400000u);
    const int held = e < kMxScaleMin ? kMxScaleMin : (e > kMxScaleMax ? kMxScaleMax : e);
    return amax >= 0x7F800000u ? 255u : (uint32_t)held;
}

// A block of 32 values -> its scale byte and 16 bytes of codes. The conversion instruction divides
// by a power of two, rounds to nearest even and saturates. sr: the stochastic draws of block t in
// direction d.
template <bool SR>
__device__ __forceinline__ uint32_t mx4_block(const float *v, uint64_t t, uint32_t d, uint32_t seed_lo,
                                              uint32_t seed_hi, u32x4_t *codes)
{
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        amax = b > amax ? b : amax;
    }
    const uint32_t e = mx4_scale(amax);
    if constexpr (!SR) {
        const float scale = __uint_as_float((e == 255 ? 127u : e) << 23);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t c = 0;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[8 * w], v[8 * w + 1], scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[8 * w + 2], v[8 * w + 3], scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[8 * w + 4], v[8 * w + 5], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[8 * w + 6], v[8 * w + 7], scale, 3);
            (*codes)[w] = e == 255 ? 0u : c;
        }
    } else {
        const float inverse = __uint_as_float((254u - (e == 255 ? 127u : e)) << 23);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint64_t n = 4 * t + w;
            const Philox4 r = philox4x32_10((uint32_t)n, (uint32_t)(n >> 32), d, 0u, seed_lo, seed_hi);
            uint32_t c = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float x = v[8 * w + j];
                const uint32_t u16 = (r.v[j / 2] >> (16 * (j % 2))) & 0xFFFFu;
                c |= (grid_sr<kFP4>(__builtin_fabsf(x) * inverse, u16) | (__float_as_uint(x) >> 31 << 3)) << (4 * j);
            }
            (*codes)[w] = e == 255 ? 0u : c;
        }
    }
    return e;
}

__device__ __forceinline__ float sigmoid(float g)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
}

} // namespace mq
