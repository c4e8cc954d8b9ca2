// mq_mx4_device.hpp -- device helpers of the microscaled 4-bit linear layers (gfx950).
#pragma once

#include "mq_device.hpp"
#include "mq_mx4.hpp"

namespace mq {

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

template <int I> struct Int {
    static constexpr int value = I;
};

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

__device__ __forceinline__ float sigmoid(float g)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g));
}
__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

// The 16 bytes of one block as an operand of a scaled product.
__device__ __forceinline__ i32x8_t operand(u32x4_t c)
{
    return i32x8_t{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

// 32x32x64: lane (row n, half h) brings the 32 elements of one block of its row, whose scale is
// byte S of its word of scales.
template <int S>
__device__ __forceinline__ f32x16_t product(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x16_t c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, S, (int)sa, S, (int)sb);
}

// Eight elements of a row of `cols` from column c on, zeros past it. Rows may begin at any element: the
// load needs no alignment. Where a row's last eight is shorter (TAIL: cols is no multiple of 8), it is
// loaded with the elements before it and shifted once it is there, so that a thread's loads are all
// made without conditions.
template <class T> struct Eight {
    T e[8];
} __attribute__((packed, aligned(sizeof(T))));
struct Reach {
    int start, shift; // first element loaded, and how many of them lie before c
};
__device__ __forceinline__ Reach reach_of(int c, int cols)
{
    const int start = max(min(c, cols - 8), 0);
    return {start, c - start};
}
// PASS: past the caches, for what is read once and would fill them.
template <bool TAIL, bool PASS = false, class T>
__device__ __forceinline__ Eight<T> load8(const T *row, Reach at, int cols)
{
    Eight<T> x;
    if (!TAIL || cols >= 8) {
        if constexpr (PASS) {
            typedef u32x4_t Any __attribute__((aligned(2)));
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                const u32x4_t w = __builtin_nontemporal_load((const Any *)(row + at.start) + i);
                __builtin_memcpy((char *)&x + 16 * i, &w, 16);
            }
            return x;
        }
        return *(const Eight<T> *)(row + at.start);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x.e[i] = i < cols ? row[i] : (T)0;
    return x;
}
// Words of two halves, or of one float: elements e on become elements 0 on, zeros behind them.
__device__ __forceinline__ u32x4_t move_down(u32x4_t w, int e)
{
    if (e & 4) w = u32x4_t{w[2], w[3], 0, 0};
    if (e & 2) w = u32x4_t{w[1], w[2], w[3], 0};
    const int s = e & 1 ? 16 : 0;
    return u32x4_t{__builtin_amdgcn_alignbit(w[1], w[0], s), __builtin_amdgcn_alignbit(w[2], w[1], s),
                   __builtin_amdgcn_alignbit(w[3], w[2], s), w[3] >> s};
}
template <bool TAIL>
__device__ __forceinline__ Eight<uint16_t> shifted(Eight<uint16_t> x, Reach at)
{
    u32x4_t w = __builtin_bit_cast(u32x4_t, x);
    if constexpr (TAIL) w = move_down(w, at.shift & 7);
    if (at.shift >= 8) w = u32x4_t{0, 0, 0, 0};
    return __builtin_bit_cast(Eight<uint16_t>, w);
}
template <bool TAIL>
__device__ __forceinline__ Eight<float> shifted(Eight<float> x, Reach at)
{
    if constexpr (TAIL) {
#pragma unroll
        for (int by = 4; by; by /= 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) x.e[i] = at.shift & by ? (i + by < 8 ? x.e[i + by] : 0.0f) : x.e[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x.e[i] = at.shift >= 8 ? 0.0f : x.e[i];
    return x;
}
template <int DT, bool TAIL>
__device__ __forceinline__ void values8(const Eight<typename Dense<DT>::T> &x, Reach at, float *v)
{
    const Eight<typename Dense<DT>::T> y = shifted<TAIL>(x, at);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = Dense<DT>::load(y.e[i]);
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest value of the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max_u32(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true)); // lane ^ 1
    return max_u32(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true)); // lane ^ 2
}

// Bits of the largest magnitude of 8 values.
__device__ __forceinline__ uint32_t amax8(const float *v)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_u32(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// Eight codes at the scale byte e. The conversion instruction divides by a power of two, rounds to
// nearest even and saturates. SR: the draws of eighth n of the blocks (4 t + its place in block t)
// in direction d.
template <bool SR>
__device__ __forceinline__ uint32_t encode8(const float *v, uint32_t e, uint64_t n, uint32_t d, uint32_t seed_lo, uint32_t seed_hi)
{
    uint32_t c = 0;
    if constexpr (!SR) {
        const float scale = __uint_as_float((e == 255 ? 127u : e) << 23);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
    } else {
        const float inverse = __uint_as_float((254u - (e == 255 ? 127u : e)) << 23);
        const Philox4 r = philox4x32_10((uint32_t)n, (uint32_t)(n >> 32), d, 0u, seed_lo, seed_hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u16 = (r.v[j / 2] >> (16 * (j % 2))) & 0xFFFFu;
            c |= (grid_sr<kFP4>(__builtin_fabsf(v[j]) * inverse, u16) | (__float_as_uint(v[j]) >> 31 << 3)) << (4 * j);
        }
    }
    return e == 255 ? 0u : c;
}

// 16 bytes to any address, past the caches. (Written out: beside a plain store of the same, the compiler
// makes one plain store of the two. The wait keeps the data's registers until they are read.)
__device__ __forceinline__ void store_past(void *to, u32x4_t x)
{
    asm volatile("global_store_dwordx4 %0, %1, off nt\n\t"
                 "s_nop 1" ::"v"(to), "v"(x)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void put(const MatView &y, int64_t r, int c, float v)
{
    static_cast<typename Dense<DT>::T *>(y.p)[r * y.stride + c] = Dense<DT>::store(v);
}

} // namespace mq
