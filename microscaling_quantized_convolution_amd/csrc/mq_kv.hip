// mq_kv.hip -- the key/value cache in 8 bits: quantizing write (mq_kv_append) and eviction by
// accumulated attention weight (mq_kv_evict).
//
// A block is 16 tokens of one head: 16 x D codes (E4M3) under one power-of-two scale 2^(e-127).
// Both operators work block by block, a wave to each block's keys or values: whole blocks are
// read and written, so no two waves share a byte.
#include "mq_attn_device.hpp"

namespace mq {
namespace {

__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Four half-precision values of magnitude 448 or less as codes.
__device__ __forceinline__ uint32_t encode4h(f16x2_t a, f16x2_t b)
{
    typedef __attribute__((ext_vector_type(2))) short s16x2_t;
    s16x2_t w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, a, 1.0f, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, b, 1.0f, true);
    return __builtin_bit_cast(uint32_t, w);
}

// The four values of a word of codes.
__device__ __forceinline__ void decode4(uint32_t w, float *v)
{
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}

// Largest of two words' halves each, as unsigned 16-bit numbers.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b)
{
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                  __builtin_bit_cast(u16x2_t, b)));
}

// Scale byte of a block whose largest magnitude has the fp32 bits `b`: the smallest power of two
// with amax <= 1.75 * 2^8 * 2^(e-127), from the exponent and one comparison of the fraction.
__device__ __forceinline__ int scale_byte(uint32_t b)
{
    const int e = (int)(b >> 23);
    if (e == 255) return 255; // a NaN or an infinity
    const int s = e - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return s > kScaleMin ? s : kScaleMin;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// Tokens a table row of `max_pages` pages can hold.
__device__ __forceinline__ int capacity(int max_pages, int page)
{
    const int64_t c = (int64_t)max_pages * page;
    return c > INT32_MAX ? INT32_MAX : (int)c;
}

// ---- append --------------------------------------------------------------------------------
//
// code = x / 2^(e-127) in E4M3, rounded to nearest, under the smallest power of two that brings the
// block's largest magnitude to 448 or less: the cache's 8 bits are the one rounding here. A block
// that holds tokens already keeps the larger of both scales, its old codes are rounded again.
//
// One wave per touched block, head and side (keys, values). Bound by the bytes: 2 B in and 1 B
// out per element; 65536 tokens of 8 heads of 128 are 403 MB in 81 us, 4.95 TB/s (a large copy
// reaches 5.16). A step of a few tokens takes 8 us, all of it call and launch. The block's largest
// magnitude is found on the 16-bit patterns (their magnitudes order like unsigned numbers), two at
// a time, while the elements stay in registers.
// Every load is made, with the token clamped into the new ones, and what does not belong is
// cleared afterwards: loads under a condition were waited for one by one.
template <int DT, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a)
{
    const int lane = threadIdx.x & 63;
    const int job = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (job >= 2 * a.c.heads) return;
    const int cap = capacity(a.max_pages, a.c.page);
    const auto held_of = [&](int s) { return clampi(a.lens[s], 0, cap); };
    const auto first_of = [&](int s) { return clampi(a.cu[s], 0, a.total); };
    const auto new_of = [&](int s) {
        const int room = cap - held_of(s), c = clampi(a.cu[s + 1], 0, a.total) - first_of(s);
        return c < 0 ? 0 : (c < room ? c : room);
    };
    int s, index;
    if (!locate_unit(blockIdx.x, a.n, [&](int q) {
            const int h = held_of(q), c = new_of(q);
            return c ? (h + c - 1) / kKvBlock - h / kKvBlock + 1 : 0;
        }, &s, &index))
        return;
    const int held = held_of(s), count = new_of(s);
    const int start = (held / kKvBlock + index) * kKvBlock; // the block's first token
    const int lo = clampi(held - start, 0, kKvBlock);
    const int hi = held + count - start < kKvBlock ? held + count - start : kKvBlock;
    const int pi = page_of(a.c, start), page = a.table[(int64_t)s * a.max_pages + pi];
    if (page < 0 || page >= a.c.pages) return;
    const int h = job >> 1, side = job & 1;
    const int64_t blk = ((int64_t)page * a.c.heads + h) * (a.c.page / kKvBlock) +
                        slot_of(a.c, start, pi) / kKvBlock;
    const RowsView &src = side ? a.v : a.k;
    const uint16_t *rows = src.p + (int64_t)(first_of(s) - held + start) * src.ts + h * src.hs;
    uint8_t *codes = (side ? a.c.vc : a.c.kc) + blk * (kKvBlock * D);
    uint8_t *scale = (side ? a.c.vs : a.c.ks) + blk;
    const int e_held = lo ? *scale : 0;

    if (side == 0) {
        // keys: 8 elements (16 B in, 8 B out) of one token to each lane at a time
        constexpr int N = D / 32;
        u32x4_t x[N];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (i * 64 + lane) / (D / 8), part = (i * 64 + lane) % (D / 8);
            x[i] = *(const u32x4_t *)(rows + clampi(t, lo, hi - 1) * src.ts + part * 8);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (i * 64 + lane) / (D / 8);
            if (t < lo || t >= hi) x[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < 4; ++w) m = max16x2(m, x[i][w] & 0x7FFF7FFFu);
        }
        m = wave_max(max16x2(m, m >> 16) & 0xFFFFu);
        const int e_new = scale_byte(__float_as_uint(Elem<DT>::f32((uint16_t)m)));
        const int e = e_new > e_held ? e_new : e_held;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (i * 64 + lane) / (D / 8), part = (i * 64 + lane) % (D / 8);
            float v[8];
            u32x2_t *at = (u32x2_t *)(codes + t * D + part * 8);
            if (t < lo) {
                const u32x2_t was = *at;
                decode4(was[0], v);
                decode4(was[1], v + 4);
            } else {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    v[2 * w] = Elem<DT>::f32((uint16_t)x[i][w]);
                    v[2 * w + 1] = Elem<DT>::f32((uint16_t)(x[i][w] >> 16));
                }
            }
            const int by = t < lo ? e_held - e : 127 - e;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = e == 255 ? 0.0f : __builtin_amdgcn_ldexpf(v[j], by);
            *at = u32x2_t{encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7])};
        }
        if (lane == 0) *scale = (uint8_t)e;
        return;
    }

    // values: two dimensions of all 16 tokens to each lane (the block's codes lie token by token
    // within a dimension)
    constexpr int N = (D / 2 + 63) / 64;
    uint32_t x[N][kKvBlock];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pair = i * 64 + lane < D / 2 ? i * 64 + lane : 0;
#pragma unroll
        for (int t = 0; t < kKvBlock; ++t)
            x[i][t] = *(const uint32_t *)(rows + clampi(t, lo, hi - 1) * src.ts + pair * 2);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int t = 0; t < kKvBlock; ++t) {
            if (t < lo || t >= hi) x[i][t] = 0;
            m = max16x2(m, x[i][t] & 0x7FFF7FFFu);
        }
    m = wave_max(max16x2(m, m >> 16) & 0xFFFFu);
    const int e_new = scale_byte(__float_as_uint(Elem<DT>::f32((uint16_t)m)));
    const int e = e_new > e_held ? e_new : e_held;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pair = i * 64 + lane;
        if (pair >= D / 2) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            u32x4_t *at = (u32x4_t *)(codes + (pair * 2 + k) * kKvBlock);
            u32x4_t was = {0, 0, 0, 0}, out;
            if (lo) was = *at;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                float v[4];
                decode4(was[w], v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 4 * w + j;
                    const float y = Elem<DT>::f32((uint16_t)(x[i][t] >> (16 * k)));
                    v[j] = __builtin_amdgcn_ldexpf(t < lo ? v[j] : y, t < lo ? e_held - e : 127 - e);
                    if (e == 255) v[j] = 0.0f;
                }
                out[w] = encode4(v[0], v[1], v[2], v[3]);
            }
            *at = out;
        }
    }
    if (lane == 0) *scale = (uint8_t)e;
}

// ---- evict ---------------------------------------------------------------------------------

// Order of weights as unsigned numbers: NaN lowest (0), then -inf ... -0 = +0 ... +inf.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 0;
    const uint32_t b = __float_as_uint(w + 0.0f); // -0 -> +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelWaves = 16, kSelSteps = 8, kSelBins = 2 * 64 * kSelWaves;
constexpr int kSelStep = 256; // tokens a wave takes at a time, four neighbours to a lane

typedef float f32x4_dword_t __attribute__((ext_vector_type(4), aligned(4)));

// One workgroup per sequence and head finds the kept tokens. Each wave owns a contiguous stretch
// of the candidates and reads their weights once, 16 bytes to a lane and all of them on their way
// together; up to kSelSteps steps a wave (32768 tokens a workgroup) stay in LDS as keys, the rest
// of a longer sequence is read again from the caches. The key of rank `need` is found by 11-bit
// digits of its distance from the smallest key, shifted so that the largest distance just fits:
// the weights' exponents, nearly equal, then spread over the bins instead of meeting in a few.
// Once at most 64 candidates share the decided digits, one wave ranks them instead (2 x 1000
// tokens, the whole call: 14.0 -> 12.4 us). Two more passes over the keys count what each wave
// keeps and write it where it belongs. Bound by the latency of these passes (the weights are 4
// bytes a token): up to 32768 tokens, 8 sequences of 8 heads, take 26 us; 110 with 8-bit digits of the
// keys, read again in each pass, 57 with keys in LDS but loaded one after another.
__global__ void __launch_bounds__(64 * kSelWaves) kv_select_kernel(EvictArgs a)
{
    __shared__ __align__(16) uint32_t held[kSelWaves][kSelSteps * kSelStep];
    __shared__ uint32_t hist[kSelBins];
    __shared__ uint32_t part[kSelWaves][2];
    __shared__ uint32_t pick[4]; // digit, rank within it, tokens of that digit; tokens collected
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int s = blockIdx.x / a.c.heads, h = blockIdx.x % a.c.heads;
    const int len = clampi(a.lens[s], 0, capacity(a.max_pages, a.c.page));
    const int take = len < a.keep ? len : a.keep;
    const int safe = a.recent < take ? a.recent : take;
    const int cand = len - safe; // tokens that compete
    const uint32_t need = take - safe; // how many of them stay
    int32_t *kept = a.kept + (int64_t)blockIdx.x * a.keep;
    const int32_t *table = a.table + (int64_t)s * a.max_pages;
    if (h == 0 && tid == 0) a.new_lens[s] = take;
    for (int i = take + tid; i < a.keep; i += blockDim.x) kept[i] = -1;
    for (int i = tid; i < safe; i += blockDim.x) kept[need + i] = cand + i;
    if (need == 0) return;
    if ((int)need == cand) {
        for (int i = tid; i < cand; i += blockDim.x) kept[i] = i;
        return;
    }
    const int stretch = ((cand + kSelWaves - 1) / kSelWaves + kSelStep - 1) / kSelStep * kSelStep;
    const int from = wave * stretch, to = from + stretch < cand ? from + stretch : cand;
    // weights of a lane's four tokens from t on (a multiple of 4: one block), NaN past the end
    // or where there is no page
    const auto weights_at = [&](int t) -> f32x4_t {
        const float nan = __builtin_nanf("");
        if (t >= to) return f32x4_t{nan, nan, nan, nan};
        const int pi = page_of(a.c, t), page = table[pi];
        if (page < 0 || page >= a.c.pages) return f32x4_t{nan, nan, nan, nan};
        return *(const f32x4_dword_t *)(a.weights + ((int64_t)page * a.c.heads + h) * a.c.page + slot_of(a.c, t, pi));
    };
    const auto keys_of = [&](f32x4_t w) {
        return u32x4_t{weight_key(w[0]), weight_key(w[1]), weight_key(w[2]), weight_key(w[3])};
    };
    // f(keys of the lane's four tokens, the first of them), over the wave's stretch
    const auto each = [&](auto f) {
        for (int t = from; t < to; t += kSelStep) {
            u32x4_t k;
            if (t - from < kSelSteps * kSelStep)
                k = *(const u32x4_t *)&held[wave][t - from + lane * 4];
            else
                k = keys_of(weights_at(t + lane * 4));
            f(k, t + lane * 4);
        }
    };
    // smallest and largest key
    uint32_t lo = ~0u, hi = 0;
    const auto range = [&](u32x4_t k, int t) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (t + q < to && k[q] < lo) lo = k[q];
            if (t + q < to && k[q] > hi) hi = k[q];
        }
    };
    {
        f32x4_t w[kSelSteps];
#pragma unroll
        for (int i = 0; i < kSelSteps; ++i) w[i] = weights_at(from + i * kSelStep + lane * 4);
#pragma unroll
        for (int i = 0; i < kSelSteps; ++i) {
            if (from + i * kSelStep >= to) break;
            const u32x4_t k = keys_of(w[i]);
            *(u32x4_t *)&held[wave][i * kSelStep + lane * 4] = k;
            range(k, from + i * kSelStep + lane * 4);
        }
        for (int t = from + kSelSteps * kSelStep + lane * 4; t < to; t += kSelStep)
            range(keys_of(weights_at(t)), t);
    }
    lo = ~wave_max(~lo);
    hi = wave_max(hi);
    if (lane == 0) {
        part[wave][0] = lo;
        part[wave][1] = hi;
    }
    __syncthreads();
    // every wave gathers the waves' parts on its lanes
    const int peer = lane % kSelWaves;
    lo = ~wave_max(~part[peer][0]);
    hi = wave_max(part[peer][1]);
    // `bound`, the distance from lo that the token of rank need (from the largest) has; `ties` of
    // its equals stay
    uint32_t bound = 0, ties = need;
    int top = 32 - __builtin_clz((hi - lo) | 1u); // bits not yet decided
    while (top > 0) {
        const int shift = top > 11 ? top - 11 : 0;
        hist[tid] = hist[tid + kSelBins / 2] = 0;
        if (tid == 0) pick[3] = 0;
        __syncthreads();
        each([&](u32x4_t k, int t) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t d = (k[q] - lo) ^ bound; // decided bits equal: below 2^top
                if (t + q < to && (top >= 32 || d >> top == 0)) atomicAdd(&hist[d >> shift], 1u);
            }
        });
        __syncthreads();
        // two bins a lane, summed from the largest down: over the wave, then over the waves
        const uint32_t c0 = hist[2 * tid], c1 = hist[2 * tid + 1];
        const uint32_t upto = wave_prefix(c0 + c1);
        if (lane == 63) part[wave][0] = upto;
        __syncthreads();
        const uint32_t sums = wave_prefix(lane < kSelWaves ? part[lane][0] : 0); // up to each wave
        // tokens above each bin
        const uint32_t over1 = __builtin_amdgcn_readlane(sums, 63) - __builtin_amdgcn_readlane(sums, wave) +
                               __builtin_amdgcn_readlane(upto, 63) - upto;
        const uint32_t over0 = over1 + c1;
        if (over1 < ties && over1 + c1 >= ties) {
            pick[0] = 2 * tid + 1;
            pick[1] = ties - over1;
            pick[2] = c1;
        }
        if (over0 < ties && over0 + c0 >= ties) {
            pick[0] = 2 * tid;
            pick[1] = ties - over0;
            pick[2] = c0;
        }
        __syncthreads();
        bound |= pick[0] << shift;
        ties = pick[1];
        top = shift;
        if (pick[2] > 64 || top == 0) continue;
        // few enough are left for a wave to rank them, one to a lane
        const int left = (int)pick[2];
        each([&](u32x4_t k, int t) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (t + q < to && ((k[q] - lo) ^ bound) >> top == 0) {
                    const uint32_t at = atomicAdd(&pick[3], 1u);
                    if (at < 64) hist[at] = k[q] - lo; // always, if the weights hold still
                }
        });
        __syncthreads();
        if (wave == 0) {
            const uint32_t mine = hist[lane < left ? lane : 0];
            uint32_t more = 0, equal = 0;
            for (int j = 0; j < left; ++j) {
                const uint32_t d = __builtin_amdgcn_readlane(mine, j);
                more += d > mine;
                equal += d == mine;
            }
            if (more < ties && more + equal >= ties) { // lanes of one distance agree
                pick[0] = mine;
                pick[1] = ties - more;
            }
        }
        __syncthreads();
        bound = pick[0];
        ties = pick[1];
        top = 0;
    }
    bound += lo;
    uint32_t over = 0, same = 0;
    each([&](u32x4_t k, int t) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            over += __popcll(__ballot(t + q < to && k[q] > bound));
            same += __popcll(__ballot(t + q < to && k[q] == bound));
        }
    });
    if (lane == 0) { // the last reads of part[][0] lie before the loop's last barrier
        part[wave][0] = over;
        part[wave][1] = same;
    }
    __syncthreads();
    {
        const uint32_t o = wave_prefix(lane < wave ? part[peer][0] : 0);
        const uint32_t e = wave_prefix(lane < wave ? part[peer][1] : 0);
        over = __builtin_amdgcn_readlane(o, 63);
        same = __builtin_amdgcn_readlane(e, 63);
    }
    each([&](u32x4_t k, int t) {
        uint32_t so = over, ss = same; // before the lane's first token
        bool is_over[4], is_same[4];
        uint64_t any_same = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            is_over[q] = t + q < to && k[q] > bound;
            is_same[q] = t + q < to && k[q] == bound;
            const uint64_t bo = __ballot(is_over[q]);
            so += bits_below(bo);
            over += __popcll(bo);
            any_same |= __ballot(is_same[q]);
        }
        if (any_same) { // rare: the equals of the bound
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint64_t bs = __ballot(is_same[q]);
                ss += bits_below(bs);
                same += __popcll(bs);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // equals that came before take the first places among the equals that stay
            const uint32_t at = so + (ss < ties ? ss : ties); // below need, if the weights hold still
            if ((is_over[q] || (is_same[q] && ss < ties)) && at < need) kept[at] = t + q;
            so += is_over[q];
            ss += is_same[q];
        }
    });
}

// One wave per new block and head: copies the keys and values of 16 kept tokens at the largest
// of their scales, and their weights. Bound by the bytes: a kept token's key is one row, but its
// value lies with the 15 others of its old block, which comes whole: 8 sequences of up to
// 32768 tokens cut to 8192, 8 heads of 128, move 287 MB (counted) in 58 us, 4.9 TB/s (101 us with
// each block loaded only when its tokens' turn came). (Copying in the workgroup
// that found the tokens, without a second launch, left 8 of 256 CUs to do it and was no faster
// at 2 x 1000 tokens.)
template <int D>
__global__ void __launch_bounds__(256) kv_move_kernel(EvictArgs a, int blocks)
{
    constexpr int KC = (D + 63) / 64;          // 16-byte pieces of keys to a lane
    constexpr int VC = (D / 2 + 63) / 64;      // pairs of dimensions of values to a lane
    const int lane = threadIdx.x & 63;
    const int h = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (h >= a.c.heads) return;
    const int s = blockIdx.x / blocks, start = blockIdx.x % blocks * kKvBlock;
    const int pn = page_of(a.c, start);
    const int to = a.new_table[(int64_t)s * a.new_max_pages + pn];
    int t = -1; // lane i < 16: the i-th token's old position
    if (lane < kKvBlock && start + lane < a.keep) t = a.kept[((int64_t)s * a.c.heads + h) * a.keep + start + lane];
    const int len = clampi(a.lens[s], 0, capacity(a.max_pages, a.c.page));
    const int take = len < a.keep ? len : a.keep;
    if (start >= take || to < 0 || to >= a.c.pages) return;
    const int hi = take - start < kKvBlock ? take - start : kKvBlock;
    const int per = a.c.page / kKvBlock;
    const int64_t blk = ((int64_t)to * a.c.heads + h) * per + slot_of(a.c, start, pn) / kKvBlock;
    int64_t from = -1; // the token's old block
    int slot = 0;      // and its slot there
    if (t >= 0 && t < len) {
        const int pi = page_of(a.c, t), page = a.table[(int64_t)s * a.max_pages + pi];
        if (page >= 0 && page < a.c.pages) {
            from = ((int64_t)page * a.c.heads + h) * per + slot_of(a.c, t, pi) / kKvBlock;
            slot = t % kKvBlock;
        }
    }
    const uint32_t live = (uint32_t)__ballot(from >= 0);
    const int64_t before = __shfl_up(from, 1);
    // tokens with which another old block begins (the kept tokens ascend)
    const uint32_t starts = (uint32_t)__ballot(from >= 0 && (lane == 0 || before != from));
    const auto block_at = [&](int i) {
        return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)from, i) |
               (int64_t)__builtin_amdgcn_readlane((int)(from >> 32), i) << 32;
    };

    // all of the keys and the first old block of the values are on their way before any is used
    u32x4_t x[KC];
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const int c = i * 64 + lane, tok = c / (D / 16), part = c % (D / 16);
        const int64_t f = __shfl(from, tok);
        const int sl = __shfl(slot, tok);
        x[i] = u32x4_t{0, 0, 0, 0};
        if (c < D && f >= 0) x[i] = *(const u32x4_t *)(a.c.kc + (f * kKvBlock + sl) * D + part * 16);
    }
    u32x4_t cur[VC][2] = {}, next[VC][2] = {};
    const auto load = [&](int i) {
        const int64_t f = block_at(i);
#pragma unroll
        for (int j = 0; j < VC; ++j)
            if (D % 128 == 0 || j * 64 + lane < D / 2) {
                const u32x4_t *p = (const u32x4_t *)(a.c.vc + (f * D + (j * 64 + lane) * 2) * kKvBlock);
                next[j][0] = p[0];
                next[j][1] = p[1];
            }
    };
    if (starts) load(__builtin_ctz(starts));
    int ek = 0, ev = 0;
    float weight = 0.0f;
    if (lane < hi) ek = ev = kScaleMin;
    if (from >= 0) {
        ek = a.c.ks[from];
        ev = a.c.vs[from];
        weight = a.weights[from * kKvBlock + slot];
    }
    if (lane < kKvBlock) a.weights[blk * kKvBlock + lane] = weight;
    const int emk = (int)wave_max((uint32_t)ek), emv = (int)wave_max((uint32_t)ev);
    if (lane == 0) {
        a.c.ks[blk] = (uint8_t)emk;
        a.c.vs[blk] = (uint8_t)emv;
    }
    // A token whose scale is smaller than the new block's is rescaled: decoded to half precision,
    // times 2^(e_src - e), encoded again. The half holds every product that is not far below the
    // smallest code exactly, so the encoding rounds once.
    const float byk = __builtin_amdgcn_ldexpf(1.0f, ek - emk), byv = __builtin_amdgcn_ldexpf(1.0f, ev - emv);
    const bool plain_k = !__any(lane < hi && ek != emk), plain_v = !__any(lane < hi && ev != emv);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const int c = i * 64 + lane, tok = c / (D / 16), part = c % (D / 16);
        if (!plain_k) {
            const float by = __shfl(byk, tok);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                x[i][w] = encode4h(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i][w], by, false),
                                   __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i][w], by, true));
        }
        if (emk == 255) x[i] = u32x4_t{0, 0, 0, 0};
        if (c < D) *(u32x4_t *)(a.c.kc + (blk * kKvBlock + tok) * D + part * 16) = x[i];
    }

    // values: a lane holds pairs of dimensions, 16 bytes of a block each. Each old block is
    // loaded once, the next one while the tokens of this one move byte by byte.
    u32x4_t out[VC][2] = {};
#pragma unroll
    for (int i = 0; i < kKvBlock; ++i) {
        if (starts >> i & 1) {
#pragma unroll
            for (int j = 0; j < VC; ++j) {
                cur[j][0] = next[j][0];
                cur[j][1] = next[j][1];
            }
            const uint32_t rest = starts & ~((2u << i) - 1);
            if (rest) load(__builtin_ctz(rest));
        }
        if (!(live >> i & 1)) continue; // stays 0
        const int sl = __builtin_amdgcn_readlane(slot, i);
        // byte sl%4 of the source word into byte i%4 of the result, the others as they are
        const uint32_t sel = (0x03020100u & ~(0xFFu << (8 * (i % 4)))) | (uint32_t)(4 + sl % 4) << (8 * (i % 4));
        const auto move = [&](int w) {
#pragma unroll
            for (int j = 0; j < VC; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    out[j][k][i / 4] = __builtin_amdgcn_perm(cur[j][k][w], out[j][k][i / 4], sel);
        };
        switch (sl / 4) { // uniform
        case 0: move(0); break;
        case 1: move(1); break;
        case 2: move(2); break;
        default: move(3);
        }
    }
    if (!plain_v) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            f16x2_t by[2];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                by[q / 2][q % 2] = (_Float16)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(byv), 4 * w + q));
#pragma unroll
            for (int j = 0; j < VC; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    out[j][k][w] = encode4h(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(out[j][k][w], 1.0f, false) * by[0],
                                            __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(out[j][k][w], 1.0f, true) * by[1]);
        }
    }
#pragma unroll
    for (int j = 0; j < VC; ++j) {
        const int pair = j * 64 + lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (emv == 255) out[j][k] = u32x4_t{0, 0, 0, 0};
            if (pair < D / 2) *(u32x4_t *)(a.c.vc + (blk * D + pair * 2 + k) * kKvBlock) = out[j][k];
        }
    }
}

template <int DT, int D>
hipError_t append(const AppendArgs &a, hipStream_t st)
{
    // blocks touched: at most one per new token, and floor(new / 16) + 2 per sequence
    int64_t units = a.total / kKvBlock + 2 * (int64_t)a.n;
    if (units > a.total) units = a.total;
    if (units == 0) return hipSuccess;
    const int64_t jobs = (2 * (int64_t)a.c.heads + 3) / 4;
    if (units > INT32_MAX || jobs > 65535) return hipErrorInvalidValue;
    kv_append_kernel<DT, D><<<dim3((unsigned)units, (unsigned)jobs), 256, 0, st>>>(a);
    return hipGetLastError();
}

template <int DT>
hipError_t append_dim(const AppendArgs &a, int d, hipStream_t st)
{
    switch (d) {
    case 64: return append<DT, 64>(a, st);
    case 96: return append<DT, 96>(a, st);
    case 128: return append<DT, 128>(a, st);
    case 192: return append<DT, 192>(a, st);
    case 256: return append<DT, 256>(a, st);
    }
    return hipErrorInvalidValue;
}

template <int D>
hipError_t evict(const EvictArgs &a, hipStream_t st)
{
    const int64_t pairs = (int64_t)a.n * a.c.heads, blocks = ((int64_t)a.keep + kKvBlock - 1) / kKvBlock;
    const int64_t jobs = ((int64_t)a.c.heads + 3) / 4;
    if (pairs > INT32_MAX || blocks * a.n > INT32_MAX || jobs > 65535) return hipErrorInvalidValue;
    kv_select_kernel<<<(unsigned)pairs, 64 * kSelWaves, 0, st>>>(a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || blocks == 0) return err;
    kv_move_kernel<D><<<dim3((unsigned)(blocks * a.n), (unsigned)jobs), 256, 0, st>>>(a, (int)blocks);
    return hipGetLastError();
}

} // namespace

hipError_t launch_kv_append(const AppendArgs &a, int d, int dtype, hipStream_t st)
{
    return dtype == MQ_BF16 ? append_dim<MQ_BF16>(a, d, st) : append_dim<MQ_F16>(a, d, st);
}

hipError_t launch_kv_evict(const EvictArgs &a, int d, hipStream_t st)
{
    if (a.n == 0) return hipSuccess;
    switch (d) {
    case 64: return evict<64>(a, st);
    case 96: return evict<96>(a, st);
    case 128: return evict<128>(a, st);
    case 192: return evict<192>(a, st);
    case 256: return evict<256>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace mq
