// mq_attn_device.hpp -- device helpers of the attention and key/value cache kernels (gfx950).
#pragma once

#include "mq_attn.hpp"

namespace mq {

typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;

// The 16-bit types: DT is an mq_dtype.
template <int DT> struct Elem;
template <> struct Elem<MQ_BF16> {
    typedef bf16x8_t x8;
    static __device__ __forceinline__ float f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    // two fp32 values rounded to nearest even, the first in the low half
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const bf16x2_t v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    // two E4M3 codes of half HI of a word, exact
    template <bool HI> static __device__ __forceinline__ uint32_t decode(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
    static __device__ __forceinline__ f32x4_t mfma16(x8 a, x8 b, f32x4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16_t mfma32(x8 a, x8 b, f32x16_t c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Elem<MQ_F16> {
    typedef f16x8_t x8;
    static __device__ __forceinline__ float f32(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const f16x2_t v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
    template <bool HI> static __device__ __forceinline__ uint32_t decode(uint32_t w)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
    }
    static __device__ __forceinline__ f32x4_t mfma16(x8 a, x8 b, f32x4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16_t mfma32(x8 a, x8 b, f32x16_t c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

// Eight E4M3 codes (two words) as an operand of 8 16-bit values, exact.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::x8 decode8(uint32_t w0, uint32_t w1)
{
    const u32x4_t v = {Elem<DT>::template decode<false>(w0), Elem<DT>::template decode<true>(w0),
                       Elem<DT>::template decode<false>(w1), Elem<DT>::template decode<true>(w1)};
    return __builtin_bit_cast(typename Elem<DT>::x8, v);
}

// Page of a table's row that holds position t >= 0, and the slot in it.
__device__ __forceinline__ int page_of(const KvView &c, int t)
{
    return (int)((uint64_t)(uint32_t)t * c.page_mul >> (31 + c.page_shift));
}
__device__ __forceinline__ int slot_of(const KvView &c, int t, int page) { return t - page * c.page; }

// Inclusive prefix sum over the wave's lanes (data-parallel moves within rows of 16 lanes, then
// the rows' last lanes to the rows behind them).
__device__ __forceinline__ int wave_prefix(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false); // 1 lane up within a row
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false); // lane 15 of a row to the next
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false); // lane 31 to the upper half
    return v;
}

// Largest unsigned value of the wave, uniform.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    const auto step = [&](uint32_t o) { v = o > v ? o : v; };
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
    step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Set bits of a lane mask below this lane.
__device__ __forceinline__ uint32_t bits_below(uint64_t m)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Where unit `unit` lies when sequences 0..n-1 own count(s) >= 0 units each, in order: false if
// it is past the last. The wave searches together, 64 sequences a step (one load each, a prefix
// sum over the lanes), so ragged batches need no table from the host. The result is uniform.
template <class Count>
__device__ __forceinline__ bool locate_unit(int unit, int n, Count count, int *seq, int *index)
{
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < n; base += 64) {
        const int c = base + lane < n ? count(base + lane) : 0;
        const int incl = wave_prefix(c);
        const uint64_t past = __ballot(incl > unit);
        if (past) {
            const int f = __builtin_ctzll(past);
            *seq = base + f;
            *index = unit - __builtin_amdgcn_readlane(incl - c, f);
            return true;
        }
        unit -= __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

} // namespace mq
