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
// (global_load_lds, no registers between) while this one is multiplied, and the first product of
// the next tile runs beside this one's softmax.
//
// Bound by the matrix instructions, and by power: 2 x 8192 tokens, 32 query heads on 8 of 128, are
// 1.10 TFLOP in 1.05 to 1.11 ms from box to box (f16 1.12 to 1.18), 990 to 1050 TFLOP/s, where a
// product of 8192 x 8192 matrices reaches 1260. The matrix units are busy for 54% of the cycles,
// the vector units for another 54%, and the clock falls to 1.8 GHz. 8 prompts of up to 2047 tokens
// (69 GFLOP) take 96 to 104 us: the last tiles leave CUs idle, and the diagonal ones are half
// masked. 32 rows to a wave let one operand read serve 32x32x16 products at two workgroups a CU; of
// 256 threads each, they cover each other's barriers.
//
// P is rounded to dtype because the second product takes 16-bit operands; m, l and O stay in fp32,
// and l sums P before it is rounded. bf16: relative error 2^-8 at any size. f16: 2^-11 down to 2^-14
// and steps of 2^-24 below, so P is held large: it is 2^11 where a score equals m, and m follows the
// tiles' largest scores down as well as up (see Range). A token's P is then off by 2^-11 of itself
// or 2^-28 of the largest P of its tile and row, whichever is more. Errors against 64 bits are 0.0020
// in bf16 and 0.00022 in f16, where rounding the output alone makes 0.0016 and 0.00019. A second
// part of P reaches that, for half as many matrix instructions again: 2 x 8192 tokens 1.41 ms in
// place of 1.05, 8 of up to 2047 120 us in place of 96. It is not taken.
#include "mq_attn_device.hpp"

#include <cfloat>
#include <cmath>
#include <type_traits>

namespace mq {
namespace {

constexpr int kM = 128, kN = 64;

// A tile of keys or values in LDS: kN rows of D/8 pieces of 16 bytes, not padded (a wave writes
// 1 KB of them at a time). The pieces of a row change places instead, by an exclusive or of their
// number with some bits of the row's: 16 rows' pieces of one number (keys, read 16 bytes a lane)
// and 4 rows' groups of four pieces (values, read 8 bytes a lane) then lie in different banks.
// The bits stay within `span` bytes, to which every row is aligned, so an address splits into
// (lane's part ^ low part of the offset) + rest.
template <int D> struct Place {
    static constexpr int kspan = D % 128 == 0 ? 256 : (D % 64 == 0 ? 128 : 64);
    static constexpr int vspan = kspan;
    static __device__ __forceinline__ int key(int row)
    {
        return D % 128 == 0 ? row & 15 : (D % 64 == 0 ? row / 2 & 7 : row / 4 & 3);
    }
    static __device__ __forceinline__ int value(int row)
    {
        return D % 128 == 0 ? (row & 3) << 2 : (D % 64 == 0 ? (row / 2 & 1) << 2 : 0);
    }
};

typedef __attribute__((ext_vector_type(8))) short s16x8_t;

// Eight elements of a key from dimension 16c + 8hh on; `at`: the lane's row of the tile at c = 0.
template <int D>
__device__ __forceinline__ u32x4_t read_k(uint32_t at, int c)
{
    typedef const __attribute__((address_space(3))) u32x4_t *lp;
    constexpr int S = Place<D>::kspan;
    return *(lp)(uintptr_t)((at ^ (uint32_t)(c * 32 % S)) + c * 32 / S * S);
}

// V's operand of 16 tokens (step u) and 32 dimensions (block i): lane (column n = dimension, half
// hh) receives tokens 4hh .. 4hh+3 and 8+4hh .. 8+4hh+3. The lane's own read, at u = i = 0, is
// `at`: token 4hh + (n%16)/4, dimensions 16(n/16) + 4(n%4) onwards.
template <int D>
__device__ __forceinline__ s16x8_t read_v(uint32_t at, int u, int i)
{
    typedef __attribute__((address_space(3))) s16x4_t *lp;
    constexpr int S = Place<D>::vspan;
    const uint32_t x = (at ^ (uint32_t)(i * 64 % S)) + i * 64 / S * S + u * 32 * D;
    const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)x);
    const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)(x + 16 * D));
    return __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Bits of a 16-bit value's exponent: all set in a NaN or an infinity.
template <int DT> constexpr uint32_t kExp = DT == MQ_BF16 ? 0x7F80u : 0x7C00u;

// The second product where V may hold a NaN or an infinity and some tokens are masked: 0 times
// such a value would reach rows that do not see it. The finite part goes the usual way (a finite
// V gives the usual bits); the rest is counted per row and dimension over the tokens that the row
// sees, with 1 for each +inf, 128 for each -inf and 16384 for each NaN (64 tokens at most: the
// sums do not mix), and added as what it amounts to. `sees`: bit j of lane (n, hh) stands for the
// j-th of its 32 tokens.
template <int DT, int D>
__device__ __forceinline__ void odd_product(uint32_t at, const typename Elem<DT>::x8 *p, uint32_t sees,
                                            f32x16_t *o)
{
    typedef typename Elem<DT>::x8 x8;
    const uint32_t codes[3] = {Elem<DT>::pack(1.0f, 0.0f), Elem<DT>::pack(128.0f, 0.0f),
                               Elem<DT>::pack(16384.0f, 0.0f)};
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        f32x16_t odd;
#pragma unroll
        for (int r = 0; r < 16; ++r) odd[r] = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s16x8_t v = read_v<D>(at, u, i), w, one;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = (uint16_t)v[j];
                const bool bad = (b & kExp<DT>) == kExp<DT>;
                const uint32_t c = (b & 0x7FFFu) > kExp<DT> ? codes[2] : (b >> 15 ? codes[1] : codes[0]);
                w[j] = (short)(bad ? c : 0u);
                v[j] = bad ? (short)0 : v[j];
                one[j] = (short)(sees >> (8 * u + j) & 1u ? codes[0] : 0u);
            }
            o[i] = Elem<DT>::mfma32(__builtin_bit_cast(x8, v), p[u], o[i]);
            odd = Elem<DT>::mfma32(__builtin_bit_cast(x8, w), __builtin_bit_cast(x8, one), odd);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int c = (int)odd[r];
            if (c & 127) o[i][r] += INFINITY;
            if (c >> 7 & 127) o[i][r] -= INFINITY;
            if (c >> 14) o[i][r] = __builtin_nanf("");
        }
    }
}

// Where P lies for each type, in powers of two; P is 2^bias where a score equals m.
//   grow   m follows a tile's largest score up where that exceeds it by more
//   fall   and down where that stays below it by more (f16 alone: bf16 has the range of fp32)
//   span   but not past this much below the row's largest score: P stays a factor of 2^span below
//          its peak in fp32 (O at most 2^(span + grow + bias + 16) times the tokens), and what lies
//          further down is less than the smallest f16 even with the largest values
// f16: P reaches 2^(grow + bias) = 2^15, below its largest number.
template <int DT> struct Range {
    static constexpr float grow = DT == MQ_F16 ? 4.0f : 8.0f, bias = DT == MQ_F16 ? 11.0f : 0.0f;
    static constexpr float fall = 8.0f, span = 64.0f;
};

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
    constexpr int KS = D / 16, DT32 = D / 32, CH = D / 8, TILE = kN * D * 2;
    constexpr int LOADS = kN * CH / 256; // 1 KB pieces of a tile to each wave
    __shared__ __align__(256) uint16_t ks[2][kN * D], vs[2][kN * D];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, hh = lane >> 5;
    // neighbouring workgroups go to different XCDs: those of one key/value head come to the same
    // one (with 8 heads), whose L2 then serves its keys and values
    const int group = a.q_heads / a.kv_heads;
    const int kvh = blockIdx.x % a.kv_heads, h = kvh * group + blockIdx.x / a.kv_heads % group;
    const auto rows_of = [&](int q, int *first) {
        const int f = a.cu[q], l = a.cu[q + 1];
        *first = f < 0 ? 0 : (f > a.total ? a.total : f);
        const int c = (l > a.total ? a.total : l) - *first;
        return c > a.max_len ? a.max_len : c;
    };
    int s, tile, first;
    const int unit = blockIdx.x / a.q_heads;
    if (a.search) { // sequence by sequence, the longest rows of each first
        int index;
        if (!locate_unit(unit, a.n, [&](int q) {
                const int c = rows_of(q, &first);
                return c > 0 ? (c + kM - 1) / kM : 0;
            }, &s, &index))
            return;
        tile = (rows_of(s, &first) + kM - 1) / kM - 1 - index;
    } else { // the longest rows of all sequences first; a shorter sequence has no such tile
        s = unit % a.n;
        tile = (a.max_len + kM - 1) / kM - 1 - unit / a.n;
    }
    const int count = rows_of(s, &first);
    if (tile * kM >= count) return;
    const int row = tile * kM + wave * 32 + n;
    const int end = (tile + 1) * kM < count ? (tile + 1) * kM : count;
    const int wave_last = tile * kM + wave * 32 + 31 < end - 1 ? tile * kM + wave * 32 + 31 : end - 1;

    // the wave's share of a tile: its 1 KB pieces, and where each lane's 16 bytes come from
    const uint16_t *kp = a.k.p + (int64_t)first * a.k.ts + kvh * a.k.hs;
    const uint16_t *vp = a.v.p + (int64_t)first * a.v.ts + kvh * a.v.hs;
    const uint32_t lds_k = lds_address(&ks[0][0]), lds_v = lds_address(&vs[0][0]);
    const uint32_t kts = (uint32_t)a.k.ts * 2, vts = (uint32_t)a.v.ts * 2; // bytes
    uint32_t from_k[LOADS], from_v[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int piece = (wave * LOADS + i) * 64 + lane, t = piece / CH, c = piece % CH;
        from_k[i] = (uint32_t)t * kts + (c ^ Place<D>::key(t)) * 16;
        from_v[i] = (uint32_t)t * vts + (c ^ Place<D>::value(t)) * 16;
    }
    const auto stage = [&](const uint16_t *p, int64_t ts, const uint32_t *from, uint32_t lds, int i) {
        if (i * kN >= end) return;
        const uint16_t *at = p + (int64_t)(i * kN) * ts;
        const uint32_t to = lds + (i & 1) * TILE + wave * LOADS * 1024;
        const int last = count - 1 - i * kN;
        if (last >= kN - 1) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j) load_to_lds(at, from[j], to + j * 1024);
        } else { // past the last token, the last one again
#pragma unroll
            for (int j = 0; j < LOADS; ++j) {
                const int t = ((wave * LOADS + j) * 64 + lane) / CH;
                load_to_lds(at, from[j] - (t > last ? (uint32_t)(t - last) * (uint32_t)(ts * 2) : 0u), to + j * 1024);
            }
        }
    };
    const auto stage_k = [&](int i) { stage(kp, a.k.ts, from_k, lds_k, i); };
    const auto stage_v = [&](int i) { stage(vp, a.v.ts, from_v, lds_v, i); };
    // the lane's places in a tile
    const uint32_t at_k = (lds_k + n * (2 * D) + hh * 16) ^ (Place<D>::key(n) * 16);
    const int tv = hh * 4 + (n & 15) / 4, dv = (n >> 4) * 16 + (n & 3) * 4;
    const uint32_t at_v = (lds_v + tv * (2 * D) + dv * 2) ^ (Place<D>::value(tv) * 16);

    x8 q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int r = row < count ? row : count - 1;
        const u32x4_t v = *(const u32x4_t *)(a.q.p + (int64_t)(first + r) * a.q.ts + h * a.q.hs + i * 16 + hh * 8);
        q[i] = __builtin_bit_cast(x8, v ^ a.q_flip);
    }
    f32x16_t o[DT32];
    float m, l, peak; // peak (f16): the row's largest score so far
    const auto begin = [&] {
#pragma unroll
        for (int d = 0; d < DT32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
        m = peak = -INFINITY;
        l = 0.0f;
        stage_k(0);
        stage_v(0);
        stage_k(1);
        lds_barrier();
    };
    // S^T of tile i
    const auto scores = [&](int i, f32x16_t *sc) {
        const uint32_t at = at_k + (i & 1) * TILE;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int r = 0; r < 16; ++r) sc[b][r] = 0.0f;
#pragma unroll
            for (int c = 0; c < KS; ++c)
                sc[b] = Elem<DT>::mfma32(__builtin_bit_cast(x8, read_k<D>(at + b * 64 * D, c)), q[c], sc[b]);
        }
    };
    // place j of 32 in a lane's scores: its token of the tile
    const auto token = [&](int b, int r) { return b * 32 + 8 * (r / 4) + 4 * hh + r % 4; };
    // scores of tile i -> p, 16 tokens each; m, l and o follow
    const auto softmax = [&](int i, auto masked, f32x16_t *sc, x8 *p) {
        if (masked) { // tokens after some of the wave's rows
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (i * kN + token(b, r) > row) sc[b][r] = -INFINITY;
        }
        float top = DT == MQ_F16 ? -INFINITY : m;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, sc[b][r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        // m follows the largest score only where that has grown by more than 2^grow in p (or is the
        // first): until then p stays in range and nothing need be rescaled
        bool moved = (top - m) * a.scale_log2e > Range<DT>::grow || (m == -INFINITY && top > m);
        if constexpr (DT == MQ_F16) {
            peak = fmaxf(peak, top);
            moved |= (m - top) * a.scale_log2e > Range<DT>::fall && (peak - top) * a.scale_log2e < Range<DT>::span;
        }
        if (__any(moved)) {
            const float was = m;
            if (moved) m = top; // row by row: no row's bits depend on another's scores
            const float keep = moved ? __builtin_amdgcn_exp2f((was - m) * a.scale_log2e) : 1.0f;
            l *= keep;
#pragma unroll
            for (int d = 0; d < DT32; ++d) o[d] *= keep;
        }
        const float base = m == -INFINITY ? 0.0f : m * a.scale_log2e - Range<DT>::bias;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            u32x4_t pw;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u / 2][u % 2 * 8 + 2 * j], a.scale_log2e, -base));
                const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u / 2][u % 2 * 8 + 2 * j + 1], a.scale_log2e, -base));
                l += p0;
                l += p1;
                pw[j] = Elem<DT>::pack(p0, p1);
            }
            p[u] = __builtin_bit_cast(x8, pw);
        }
    };

    // Tile i, whose scores are in sc, which then holds those of tile i + 1: the first product of
    // the next tile keeps the matrix unit busy under this one's softmax.
    f32x16_t sc[2];
    const auto step = [&](int i, auto masked) {
        lds_barrier(); // K of tile i + 1 and V of tile i are there; tile i - 1 is no longer read
        stage_k(i + 2);
        stage_v(i + 1);
        f32x16_t cur[2] = {sc[0], sc[1]};
        if (!masked || (i + 1) * kN <= wave_last) scores(i + 1, sc);
        if (masked && i * kN > wave_last) return; // past the wave's rows
        x8 p[4];
        softmax(i, masked, cur, p);
        const uint32_t at = at_v + (i & 1) * TILE;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int d = 0; d < DT32; ++d)
                o[d] = Elem<DT>::mfma32(__builtin_bit_cast(x8, read_v<D>(at, u, d)), p[u], o[d]);
    };
    const int sure = tile * kM / kN; // tiles that all rows of the workgroup see
    begin();
    scores(0, sc);
    for (int i = 0; i < sure; ++i) step(i, std::false_type());
    for (int i = sure; i * kN < end; ++i) step(i, std::true_type());

    // A NaN or an infinity of V at a masked place has made some result NaN. Then, and where one
    // is due, everything is done again with the masked products taken apart.
    float odd = 0.0f;
#pragma unroll
    for (int d = 0; d < DT32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) odd = __builtin_fmaf(o[d][r], 0.0f, odd);
    if (__syncthreads_or(!(odd == 0.0f))) {
        begin();
        for (int i = 0; i * kN < end; ++i) {
            lds_barrier();
            if (i) stage_k(i + 1);
            stage_v(i + 1);
            x8 p[4];
            scores(i, sc);
            softmax(i, std::true_type(), sc, p);
            uint32_t sees = 0;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) sees |= (i * kN + token(b, r) <= row ? 1u : 0u) << (b * 16 + r);
            odd_product<DT, D>(at_v + (i & 1) * TILE, p, sees, o);
        }
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
    // One workgroup for each tile that a sequence of max_len would have, as long as at most about
    // three in four of them find nothing to do; else one for each that there can be, which
    // search for theirs. Searching against not, 32 query heads on 8 of 128, one long prompt among
    // short ones: 512 sequences (one of 4096, the others 30 tokens) 372 and 551 us, 256 (8192 and
    // 300) 1185 and 1352, 64 (8192 and 500) 819 and 836; equal prompts start earlier without.
    const int64_t direct = ((int64_t)a.max_len + kM - 1) / kM * a.n, there = (int64_t)a.total / kM + a.n;
    PromptArgs b = a;
    b.search = direct > 4 * there;
    const int64_t groups = (b.search ? there : direct) * a.q_heads;
    if (groups > INT32_MAX) return hipErrorInvalidValue;
    attn_prompt_kernel<DT, D><<<(unsigned)groups, 256, 0, st>>>(b);
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
