// mq_attn_prompt.hip -- causal attention over whole prompts, packed sequences, grouped heads.
//
// out = softmax(scale q K^T) V with a running maximum m and sum l per row: a workgroup holds 128
// query rows of one head (32 per wave) and passes over the keys 64 at a time, staged in LDS:
//   S^T = K Q^T       v_mfma 32x32x16
//   P   = 2^(S - m)   fp32, in the accumulator registers, rounded to dtype
//   O^T += V^T P^T    v_mfma 32x32x16
// S^T leaves lane (column n = row, half hh) with tokens 8i + 4hh + j of a 32-token tile; the
// second product takes its 16 tokens of a step in that same order, so P never changes lanes, and
// V's operand comes transposed out of LDS in the same order (ds_read_b64_tr_b16).
#include "mq_attn_device.hpp"

#include <cfloat>
#include <cmath>

namespace mq {
namespace {

constexpr int kM = 128, kN = 64;

typedef __attribute__((ext_vector_type(8))) short s16x8_t;

// V's operand of 16 tokens from `at` on and 32 dimensions: lane (column n = dimension, half hh)
// receives tokens 4hh .. 4hh+3 and 8+4hh .. 8+4hh+3. `at` is the lane's own address of the read:
// token 4hh + (n%16)/4, dimensions 16(n/16) + 4(n%4) onwards.
template <int LV>
__device__ __forceinline__ s16x8_t read_v(const uint16_t *at)
{
    typedef s16x4_t __attribute__((address_space(3))) *lp;
    const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)at);
    const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 8 * LV));
    return __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Bits of a 16-bit value's exponent: all set in a NaN or an infinity.
template <int DT> constexpr uint32_t kExp = DT == MQ_BF16 ? 0x7F80u : 0x7C00u;

// Any NaN or infinity among two packed values.
template <int DT> __device__ __forceinline__ bool not_finite(uint32_t w)
{
    return (w & kExp<DT>) == kExp<DT> || ((w >> 16) & kExp<DT>) == kExp<DT>;
}

// The second product where V holds a NaN or an infinity and some tokens are masked: 0 times such
// a value would reach rows that do not see it. The finite part goes the usual way; the rest is
// counted per row and dimension over the tokens that the row sees, with 1 for each +inf, 128
// for each -inf and 16384 for each NaN (64 tokens at most: the sums do not mix), and added as
// what it amounts to. `sees`: bit j of lane (n, hh) stands for the j-th of its 32 tokens.
template <int DT, int DT32, int LV>
__device__ __forceinline__ void odd_product(const uint16_t *at, const typename Elem<DT>::x8 *p,
                                            uint32_t sees, f32x16_t *o)
{
    typedef typename Elem<DT>::x8 x8;
    const uint32_t codes[3] = {Elem<DT>::pack(1.0f, 0.0f), Elem<DT>::pack(128.0f, 0.0f),
                               Elem<DT>::pack(16384.0f, 0.0f)};
    for (int i = 0; i < DT32; ++i) {
        f32x16_t odd, add;
#pragma unroll
        for (int r = 0; r < 16; ++r) odd[r] = add[r] = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s16x8_t v = read_v<LV>(at + u * 16 * LV + i * 32), w, one;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = (uint16_t)v[j];
                const bool bad = (b & kExp<DT>) == kExp<DT>;
                const uint32_t c = (b & 0x7FFFu) > kExp<DT> ? codes[2] : (b >> 15 ? codes[1] : codes[0]);
                w[j] = (short)(bad ? c : 0u);
                v[j] = bad ? (short)0 : v[j];
                one[j] = (short)(sees >> (8 * u + j) & 1u ? codes[0] : 0u);
            }
            add = Elem<DT>::mfma32(__builtin_bit_cast(x8, v), p[u], add);
            odd = Elem<DT>::mfma32(__builtin_bit_cast(x8, w), __builtin_bit_cast(x8, one), odd);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int c = (int)odd[r];
            if (c & 127) add[r] += INFINITY;
            if (c >> 7 & 127) add[r] -= INFINITY;
            if (c >> 14) add[r] = __builtin_nanf("");
        }
#pragma unroll
        for (int k = 0; k < DT32; ++k) // o is held in registers: no indexing at run time
            if (k == i) o[k] += add;
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(256, D > 128 ? 1 : 2) attn_prompt_kernel(PromptArgs a)
{
    typedef typename Elem<DT>::x8 x8;
    constexpr int KS = D / 16, DT32 = D / 32;
    constexpr int LK = D + 8;                    // rows 4 banks apart (of 64): b128 reads of 16 rows
    constexpr int LV = D % 64 == 32 ? D : D + 32; // rows 16 or 48 banks apart: 4 rows of 64 B
    __shared__ __align__(16) uint16_t ks[kN * LK], vs[kN * LV];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, hh = lane >> 5;
    const int tiles = (a.max_len + kM - 1) / kM;
    const int h = blockIdx.x % a.q_heads, s = blockIdx.x / a.q_heads % a.n;
    const int tile = tiles - 1 - (int)(blockIdx.x / a.q_heads / a.n); // the longest rows first
    int first = a.cu[s], count = a.cu[s + 1];
    first = first < 0 ? 0 : (first > a.total ? a.total : first);
    count = (count > a.total ? a.total : count) - first;
    if (count > a.max_len) count = a.max_len;
    if (tile * kM >= count) return;
    const int kvh = h / (a.q_heads / a.kv_heads);
    const int row = tile * kM + wave * 32 + n;

    x8 q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        u32x4_t v = {0, 0, 0, 0};
        if (row < count) v = *(const u32x4_t *)(a.q.p + (int64_t)(first + row) * a.q.ts + h * a.q.hs + i * 16 + hh * 8);
        q[i] = __builtin_bit_cast(x8, v ^ a.q_flip);
    }
    f32x16_t o[DT32];
#pragma unroll
    for (int i = 0; i < DT32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    const uint16_t *kp = a.k.p + (int64_t)first * a.k.ts + kvh * a.k.hs;
    const uint16_t *vp = a.v.p + (int64_t)first * a.v.ts + kvh * a.v.hs;
    const int end = (tile + 1) * kM < count ? (tile + 1) * kM : count;

    for (int t0 = 0; t0 < end; t0 += kN) {
        __syncthreads();
        constexpr int CH = D / 8;
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kN * CH / 256; ++i) {
            const int c = i * 256 + tid, t = c / CH, part = c % CH;
            u32x4_t kv = {0, 0, 0, 0}, vv = {0, 0, 0, 0};
            if (t0 + t < count) {
                kv = *(const u32x4_t *)(kp + (int64_t)(t0 + t) * a.k.ts + part * 8);
                vv = *(const u32x4_t *)(vp + (int64_t)(t0 + t) * a.v.ts + part * 8);
            }
            *(u32x4_t *)&ks[t * LK + part * 8] = kv;
            *(u32x4_t *)&vs[t * LV + part * 8] = vv;
#pragma unroll
            for (int w = 0; w < 4; ++w) odd |= not_finite<DT>(vv[w]);
        }
        const bool masked = t0 + kN > tile * kM; // some row of the workgroup does not see all tokens
        if (masked)
            odd = __syncthreads_or(odd);
        else
            __syncthreads();
        if (t0 > tile * kM + wave * 32 + 31) continue; // past this wave's last row
        f32x16_t sc[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[b][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const x8 k = *(const x8 *)&ks[(b * 32 + n) * LK + i * 16 + hh * 8];
                sc[b] = Elem<DT>::mfma32(k, q[i], sc[b]);
            }
        }
        if (t0 + kN > tile * kM + wave * 32) { // tokens after some of the wave's rows
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (t0 + b * 32 + 8 * (r / 4) + 4 * hh + r % 4 > row) sc[b][r] = -INFINITY;
        }
        float top = m;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[b][r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : top * a.scale_log2e;
        const float keep = __builtin_amdgcn_exp2f(__builtin_fmaf(m, a.scale_log2e, -base));
        m = top;
        l *= keep;
#pragma unroll
        for (int i = 0; i < DT32; ++i) o[i] *= keep;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                sc[b][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][r], a.scale_log2e, -base));
                l += sc[b][r];
            }
        x8 p[4]; // 16 tokens each
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            u32x4_t pw;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                pw[j] = Elem<DT>::pack(sc[u / 2][u % 2 * 8 + 2 * j], sc[u / 2][u % 2 * 8 + 2 * j + 1]);
            p[u] = __builtin_bit_cast(x8, pw);
        }
        const uint16_t *at = &vs[(hh * 4 + (n & 15) / 4) * LV + (n >> 4) * 16 + (n & 3) * 4];
        if (masked && odd) {
            uint32_t sees = 0;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sees |= (t0 + b * 32 + 8 * (r / 4) + 4 * hh + r % 4 <= row ? 1u : 0u) << (b * 16 + r);
            odd_product<DT, DT32, LV>(at, p, sees, o);
            continue;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < DT32; ++i)
                o[i] = Elem<DT>::mfma32(__builtin_bit_cast(x8, read_v<LV>(at + u * 16 * LV + i * 32)), p[u], o[i]);
    }
    l += __shfl_xor(l, 32);
    if (row >= count) return;
    const float inv = 1.0f / l;
    uint16_t *dst = a.out + (int64_t)(first + row) * a.out_ts + h * a.out_hs;
#pragma unroll
    for (int i = 0; i < DT32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            *(u32x2_t *)(dst + i * 32 + 2 * r + hh * 4) =
                u32x2_t{Elem<DT>::pack(o[i][r] * inv, o[i][r + 1] * inv),
                        Elem<DT>::pack(o[i][r + 2] * inv, o[i][r + 3] * inv)};
}

template <int DT, int D>
hipError_t prompt(const PromptArgs &a, hipStream_t st)
{
    const int64_t tiles = ((int64_t)a.max_len + kM - 1) / kM;
    const int64_t groups = tiles * a.n * a.q_heads;
    if (groups > INT32_MAX) return hipErrorInvalidValue;
    attn_prompt_kernel<DT, D><<<(unsigned)groups, 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t prompt_dim(const PromptArgs &a, int d, hipStream_t st)
{
    switch (d) {
    case 64: return prompt<DT, 64>(a, st);
    case 96: return prompt<DT, 96>(a, st);
    case 128: return prompt<DT, 128>(a, st);
    case 192: return prompt<DT, 192>(a, st);
    case 256: return prompt<DT, 256>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace

hipError_t launch_attn_prompt(const PromptArgs &args, int d, int dtype, hipStream_t st)
{
    PromptArgs a = args;
    if (a.n == 0 || a.total == 0 || a.max_len == 0) return hipSuccess;
    // the kernel takes the largest score before it scales, and masks with -inf: a negative scale
    // goes into q's sign, and 0 becomes the smallest normal number
    a.q_flip = a.scale_log2e < 0.0f ? 0x80008000u : 0u;
    a.scale_log2e = fabsf(a.scale_log2e);
    if (a.scale_log2e < FLT_MIN) a.scale_log2e = FLT_MIN;
    return dtype == MQ_BF16 ? prompt_dim<MQ_BF16>(a, d, st) : prompt_dim<MQ_F16>(a, d, st);
}

} // namespace mq
