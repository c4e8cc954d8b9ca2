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
// The next tile's keys and values are on their way from memory into the other half of LDS
// (global_load_lds, no registers between) while this one is multiplied.
#include "mq_attn_device.hpp"

#include <cfloat>
#include <cmath>

namespace mq {
namespace {

constexpr int kM = 128, kN = 64;

// Where 16-byte piece c of a row lies in LDS: rows are not padded (a wave writes 1 KB of them at
// a time), the pieces of a row change places instead, so that 16 rows' pieces of one number
// (keys, read 16 bytes a lane) and 4 rows' groups of four pieces (values, read 8 bytes a lane)
// lie in different banks.
template <int D> __device__ __forceinline__ int key_place(int row, int c)
{
    return c ^ (D == 64 || D == 192 ? row / 2 & 7 : (D == 96 ? row / 4 & 3 : row & 15));
}
template <int D> __device__ __forceinline__ int value_place(int row, int c)
{
    return c ^ (D == 64 || D == 192 ? (row / 2 & 1) << 2 : (D == 96 ? 0 : (row & 3) << 2));
}

typedef __attribute__((ext_vector_type(8))) short s16x8_t;

// V's operand of 16 tokens from `at` on and 32 dimensions: lane (column n = dimension, half hh)
// receives tokens 4hh .. 4hh+3 and 8+4hh .. 8+4hh+3 of step u. The lane's own read is of token
// t = 4hh + (n%16)/4, dimensions d = 16(n/16) + 4(n%4) onwards; the places of the 32 dimensions'
// four pieces depend on t%4 (or t/2%2) alone, which no step changes.
template <int D>
__device__ __forceinline__ s16x8_t read_v(const uint16_t *vt, int t, int d, int u, int i)
{
    typedef s16x4_t __attribute__((address_space(3))) *lp;
    const uint16_t *at = vt + (u * 16 + t) * D + value_place<D>(t, i * 4 + d / 8) * 8 + d % 8;
    const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)at);
    const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(at + 8 * D));
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
template <int DT, int D>
__device__ __forceinline__ void odd_product(const uint16_t *vt, int tv, int dv, const typename Elem<DT>::x8 *p,
                                            uint32_t sees, f32x16_t *o)
{
    typedef typename Elem<DT>::x8 x8;
    constexpr int DT32 = D / 32;
    const uint32_t codes[3] = {Elem<DT>::pack(1.0f, 0.0f), Elem<DT>::pack(128.0f, 0.0f),
                               Elem<DT>::pack(16384.0f, 0.0f)};
    for (int i = 0; i < DT32; ++i) {
        f32x16_t odd, add;
#pragma unroll
        for (int r = 0; r < 16; ++r) odd[r] = add[r] = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s16x8_t v = read_v<D>(vt, tv, dv, u, i), w, one;
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

// 64 lanes x 16 bytes from base + off (bytes, per lane) to 1 KB of LDS at byte `lds`. The caller
// waits (vmcnt) before the data is read. Nothing is returned in registers.
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory");
}

// Every load into LDS has arrived, every read of LDS is done, for all waves.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\t"
                 "s_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

template <int DT, int D>
__global__ void __launch_bounds__(256, D > 128 ? 1 : 2) attn_prompt_kernel(PromptArgs a)
{
    typedef typename Elem<DT>::x8 x8;
    constexpr int KS = D / 16, DT32 = D / 32, CH = D / 8;
    constexpr int LOADS = kN * CH / 256; // 1 KB pieces of a tile to each wave
    __shared__ __align__(16) uint16_t ks[2][kN * D], vs[2][kN * D];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, hh = lane >> 5;
    const int tiles = (a.max_len + kM - 1) / kM;
    // neighbouring workgroups go to different XCDs: those of one key/value head come to the same
    // one (with 8 heads), whose L2 then serves its keys and values
    const int group = a.q_heads / a.kv_heads;
    const int kvh = blockIdx.x % a.kv_heads, h = kvh * group + blockIdx.x / a.kv_heads % group;
    const int s = blockIdx.x / a.q_heads % a.n;
    const int tile = tiles - 1 - (int)(blockIdx.x / a.q_heads / a.n); // the longest rows first
    int first = a.cu[s], count = a.cu[s + 1];
    first = first < 0 ? 0 : (first > a.total ? a.total : first);
    count = (count > a.total ? a.total : count) - first;
    if (count > a.max_len) count = a.max_len;
    if (tile * kM >= count) return;
    const int row = tile * kM + wave * 32 + n;
    const int end = (tile + 1) * kM < count ? (tile + 1) * kM : count;

    const uint16_t *kp = a.k.p + (int64_t)first * a.k.ts + kvh * a.k.hs;
    const uint16_t *vp = a.v.p + (int64_t)first * a.v.ts + kvh * a.v.hs;
    const uint32_t lds_k = lds_address(&ks[0][0]), lds_v = lds_address(&vs[0][0]);
    const auto stage = [&](int t0, int buf) { // past the last token, the last one again
        const uint16_t *kt = kp + (int64_t)t0 * a.k.ts, *vt = vp + (int64_t)t0 * a.v.ts;
        const int last = count - 1 - t0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int piece = (wave * LOADS + i) * 64 + lane, t = piece / CH, c = piece % CH;
            const int from = t < last ? t : last;
            const uint32_t to = (uint32_t)(buf * kN * D * 2 + (wave * LOADS + i) * 1024);
            load_to_lds(kt, (uint32_t)from * (uint32_t)(a.k.ts * 2) + key_place<D>(t, c) * 16, lds_k + to);
            load_to_lds(vt, (uint32_t)from * (uint32_t)(a.v.ts * 2) + value_place<D>(t, c) * 16, lds_v + to);
        }
    };

    x8 q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        u32x4_t v = {0, 0, 0, 0};
        if (row < count) v = *(const u32x4_t *)(a.q.p + (int64_t)(first + row) * a.q.ts + h * a.q.hs + i * 16 + hh * 8);
        q[i] = __builtin_bit_cast(x8, v ^ a.q_flip);
    }
    stage(0, 0);
    f32x16_t o[DT32];
#pragma unroll
    for (int i = 0; i < DT32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    lds_barrier();

    int buf = 0;
    for (int t0 = 0; t0 < end; t0 += kN, buf ^= 1) {
        if (t0) lds_barrier();
        if (t0 + kN < end) stage(t0 + kN, buf ^ 1);
        const uint16_t *kt = ks[buf], *vt = vs[buf];
        const bool masked = t0 + kN > tile * kM; // some row of the workgroup does not see all tokens
        bool odd = false;
        if (masked) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const u32x4_t w = *(const u32x4_t *)&vt[(i * 256 + tid) * 8];
                odd |= not_finite<DT>(w[0]) || not_finite<DT>(w[1]) || not_finite<DT>(w[2]) || not_finite<DT>(w[3]);
            }
            odd = __syncthreads_or(odd);
        }
        if (t0 > tile * kM + wave * 32 + 31) continue; // past this wave's last row
        f32x16_t sc[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[b][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const x8 k = *(const x8 *)&kt[(b * 32 + n) * D + key_place<D>(n, i * 2 + hh) * 8];
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
        // m follows the largest score only where that has grown by a factor of 2^8 in p (or is the
        // first): until then p stays below 2^8 and nothing need be rescaled
        const bool grown = (top - m) * a.scale_log2e > 8.0f || (m == -INFINITY && top > m);
        if (__any(grown)) {
            const float was = m;
            if (grown) m = top; // row by row: no row's bits depend on another's scores
            const float keep = grown ? __builtin_amdgcn_exp2f((was - m) * a.scale_log2e) : 1.0f;
            l *= keep;
#pragma unroll
            for (int i = 0; i < DT32; ++i) o[i] *= keep;
        }
        const float base = m == -INFINITY ? 0.0f : m * a.scale_log2e;
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
        const int tv = hh * 4 + (n & 15) / 4, dv = (n >> 4) * 16 + (n & 3) * 4;
        if (masked && odd) {
            uint32_t sees = 0;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sees |= (t0 + b * 32 + 8 * (r / 4) + 4 * hh + r % 4 <= row ? 1u : 0u) << (b * 16 + r);
            odd_product<DT, D>(vt, tv, dv, p, sees, o);
            continue;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < DT32; ++i)
                o[i] = Elem<DT>::mfma32(__builtin_bit_cast(x8, read_v<D>(vt, tv, dv, u, i)), p[u], o[i]);
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
