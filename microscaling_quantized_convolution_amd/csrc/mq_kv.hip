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

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint32_t o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
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
// One wave per touched block, head and side (keys, values). Bound by the bytes: 2 B in and 1 B
// out per element. The block's largest magnitude is found on the 16-bit patterns (their
// magnitudes order like unsigned numbers), two at a time, while the elements stay in registers.
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
    const int page = a.table[(int64_t)s * a.max_pages + start / a.c.page];
    if (page < 0 || page >= a.c.pages) return;
    const int h = job >> 1, side = job & 1;
    const int64_t blk = ((int64_t)page * a.c.heads + h) * (a.c.page / kKvBlock) +
                        start % a.c.page / kKvBlock;
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
            x[i] = u32x4_t{0, 0, 0, 0};
            if (t >= lo && t < hi) x[i] = *(const u32x4_t *)(rows + t * src.ts + part * 8);
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
        const int pair = i * 64 + lane;
#pragma unroll
        for (int t = 0; t < kKvBlock; ++t) {
            x[i][t] = 0;
            if (t >= lo && t < hi && pair < D / 2)
                x[i][t] = *(const uint32_t *)(rows + t * src.ts + pair * 2);
            m = max16x2(m, x[i][t] & 0x7FFF7FFFu);
        }
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

constexpr int kSelWaves = 16, kSelKeys = 32, kSelBins = 2048;

// One workgroup per sequence and head finds the kept tokens. Each wave owns a contiguous stretch
// of the candidates and reads their weights once; up to kSelKeys keys a lane (32768 tokens a
// workgroup) stay in registers, the rest of a longer sequence is read again from the caches. The
// key of rank `need` is found by three 11-bit digits of its distance from the smallest key,
// shifted so that the largest distance just fits: the weights' exponents, nearly equal, then
// spread over the bins instead of meeting in a few. Two more passes over the keys count what each
// wave keeps and write it where it belongs.
__global__ void __launch_bounds__(64 * kSelWaves) kv_select_kernel(EvictArgs a)
{
    __shared__ uint32_t hist[kSelBins];
    __shared__ uint32_t part[kSelWaves][2];
    __shared__ uint32_t pick[2]; // digit, rank within it
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
    const int stretch = ((cand + kSelWaves - 1) / kSelWaves + 63) & ~63;
    const int from = wave * stretch, to = from + stretch < cand ? from + stretch : cand;
    const auto key_of = [&](int t) -> uint32_t {
        const int page = table[t / a.c.page];
        if (page < 0 || page >= a.c.pages) return 0;
        return weight_key(a.weights[((int64_t)page * a.c.heads + h) * a.c.page + t % a.c.page]);
    };
    uint32_t keys[kSelKeys];
#pragma unroll
    for (int j = 0; j < kSelKeys; ++j) {
        const int t = from + j * 64 + lane;
        keys[j] = t < to ? key_of(t) : 0;
    }
    // f(key, first token of the wave's 64, whether this lane has one), over the wave's stretch
    const auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kSelKeys; ++j)
            if (from + j * 64 < to) f(keys[j], from + j * 64, from + j * 64 + lane < to);
        for (int t = from + kSelKeys * 64; t < to; t += 64)
            f(t + lane < to ? key_of(t + lane) : 0, t, t + lane < to);
    };
    // smallest and largest key
    uint32_t lo = ~0u, hi = 0;
    each([&](uint32_t k, int, bool live) {
        if (live && k < lo) lo = k;
        if (live && k > hi) hi = k;
    });
    lo = ~wave_max(~lo);
    hi = wave_max(hi);
    if (lane == 0) {
        part[wave][0] = lo;
        part[wave][1] = hi;
    }
    __syncthreads();
    for (int w = 0; w < kSelWaves; ++w) {
        lo = part[w][0] < lo ? part[w][0] : lo;
        hi = part[w][1] > hi ? part[w][1] : hi;
    }
    // `bound`, the distance from lo that the token of rank need (from the largest) has; `ties` of
    // its equals stay
    uint32_t bound = 0, ties = need;
    int top = 32 - __builtin_clz((hi - lo) | 1u); // bits not yet decided
    while (top > 0) {
        const int shift = top > 11 ? top - 11 : 0;
        for (int i = tid; i < kSelBins; i += blockDim.x) hist[i] = 0;
        __syncthreads();
        each([&](uint32_t k, int, bool live) {
            const uint32_t d = (k - lo) ^ bound; // decided bits equal: below 2^top
            if (live && (top >= 32 || d >> top == 0)) atomicAdd(&hist[d >> shift], 1u);
        });
        __syncthreads();
        if (wave == 0) { // 32 bins a lane, from the largest lane down
            uint32_t sum = 0;
            for (int j = 0; j < kSelBins / 64; ++j) sum += hist[lane * (kSelBins / 64) + j];
            uint32_t above = sum; // sum over this lane and those above it
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = __shfl_down(above, d);
                if (lane + d < 64) above += o;
            }
            above -= sum;
            if (above < ties && above + sum >= ties) { // exactly one lane
                int j = kSelBins / 64 - 1;
                for (uint32_t c; above + (c = hist[lane * (kSelBins / 64) + j]) < ties; --j) above += c;
                pick[0] = lane * (kSelBins / 64) + j;
                pick[1] = ties - above;
            }
        }
        __syncthreads();
        bound |= pick[0] << shift;
        ties = pick[1];
        top = shift;
        __syncthreads();
    }
    bound += lo;
    uint32_t over = 0, same = 0;
    each([&](uint32_t k, int, bool live) {
        over += __popcll(__ballot(live && k > bound));
        same += __popcll(__ballot(live && k == bound));
    });
    if (lane == 0) {
        part[wave][0] = over;
        part[wave][1] = same;
    }
    __syncthreads();
    over = same = 0;
    for (int w = 0; w < wave; ++w) {
        over += part[w][0];
        same += part[w][1];
    }
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    each([&](uint32_t k, int t, bool live) {
        const uint64_t bo = __ballot(live && k > bound), bs = __ballot(live && k == bound);
        const uint32_t so = over + __popcll(bo & below), ss = same + __popcll(bs & below);
        // equals that came before take the first places among the equals that stay
        const bool stays = (bo >> lane & 1) || ((bs >> lane & 1) && ss < ties);
        if (stays) kept[so + (ss < ties ? ss : ties)] = t + lane;
        over += __popcll(bo);
        same += __popcll(bs);
    });
}

// One wave per new block, head and side: copies the 16 kept tokens at the largest of their
// scales, and (the wave of the keys) their weights.
template <int D>
__global__ void __launch_bounds__(256) kv_move_kernel(EvictArgs a, int blocks)
{
    const int lane = threadIdx.x & 63;
    const int job = blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (job >= 2 * a.c.heads) return;
    const int h = job >> 1, side = job & 1;
    const int s = blockIdx.x / blocks, start = blockIdx.x % blocks * kKvBlock;
    const int len = clampi(a.lens[s], 0, capacity(a.max_pages, a.c.page));
    const int take = len < a.keep ? len : a.keep;
    if (start >= take) return;
    const int hi = take - start < kKvBlock ? take - start : kKvBlock;
    const int to = a.new_table[(int64_t)s * a.new_max_pages + start / a.c.page];
    if (to < 0 || to >= a.c.pages) return;
    const int per = a.c.page / kKvBlock;
    const int64_t blk = ((int64_t)to * a.c.heads + h) * per + start % a.c.page / kKvBlock;
    uint8_t *scales = side ? a.c.vs : a.c.ks;
    uint8_t *all = side ? a.c.vc : a.c.kc;
    // lane t < 16: where token t comes from (block, slot of the block, scale byte)
    int64_t from = -1;
    int slot = 0, e_src = 0;
    if (lane < hi) {
        const int t = a.kept[((int64_t)s * a.c.heads + h) * a.keep + start + lane];
        e_src = kScaleMin;
        if (t >= 0 && t < len) {
            const int page = a.table[(int64_t)s * a.max_pages + t / a.c.page];
            if (page >= 0 && page < a.c.pages) {
                from = ((int64_t)page * a.c.heads + h) * per + t % a.c.page / kKvBlock;
                slot = t % kKvBlock;
                e_src = scales[from];
            }
        }
    }
    const int e = (int)wave_max((uint32_t)e_src);
    if (lane == 0) scales[blk] = (uint8_t)e;
    if (side == 0 && lane < kKvBlock)
        a.weights[blk * kKvBlock + lane] = from >= 0 ? a.weights[from * kKvBlock + slot] : 0.0f;
    const int by = e_src - e; // per token, on its lane

    if (side == 0) {
        constexpr int N = D / 32;
        u32x2_t x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (i * 64 + lane) / (D / 8), part = (i * 64 + lane) % (D / 8);
            const int64_t f = __shfl(from, t);
            const int sl = __shfl(slot, t);
            x[i] = u32x2_t{0, 0};
            if (f >= 0) x[i] = *(const u32x2_t *)(all + (f * kKvBlock + sl) * D + part * 8);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = (i * 64 + lane) / (D / 8), part = (i * 64 + lane) % (D / 8);
            const int b = __shfl(by, t);
            float v[8];
            decode4(x[i][0], v);
            decode4(x[i][1], v + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = e == 255 ? 0.0f : __builtin_amdgcn_ldexpf(v[j], b);
            *(u32x2_t *)(all + (blk * kKvBlock + t) * D + part * 8) =
                u32x2_t{encode4(v[0], v[1], v[2], v[3]), encode4(v[4], v[5], v[6], v[7])};
        }
        return;
    }
    // Values: a lane holds two dimensions, 16 bytes a block each. The kept tokens ascend, so those
    // of one old block come together: each old block is loaded once, the next one while the
    // tokens of this one move byte by byte (v_perm_b32, under uniform selectors).
    constexpr int N = (D / 2 + 63) / 64;
    const uint32_t starts = (uint32_t)__ballot(lane < hi && from >= 0 && (lane == 0 || from != __shfl(from, lane ? lane - 1 : 0)));
    const bool plain = !__any(lane < hi && by != 0) && e != 255;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pair = i * 64 + lane;
        if (pair >= D / 2) continue;
        const auto load = [&](int t, u32x4_t *x) {
            const int64_t f = (int64_t)((uint32_t)__builtin_amdgcn_readlane((int)from, t)) |
                              (int64_t)__builtin_amdgcn_readlane((int)(from >> 32), t) << 32;
            const u32x4_t *p = (const u32x4_t *)(all + (f * D + pair * 2) * kKvBlock);
            x[0] = p[0];
            x[1] = p[1];
        };
        u32x4_t cur[2] = {}, next[2] = {}, out[2] = {};
        if (starts) load(__builtin_ctz(starts), next);
#pragma unroll
        for (int t = 0; t < kKvBlock; ++t) {
            if (starts >> t & 1) {
                cur[0] = next[0];
                cur[1] = next[1];
                const uint32_t rest = starts & ~((2u << t) - 1);
                if (rest) load(__builtin_ctz(rest), next);
            }
            if (t >= hi || __builtin_amdgcn_readlane((int)(from >> 32), t) < 0) continue; // 0
            const int sl = __builtin_amdgcn_readlane(slot, t);
            // byte sl%4 of the source word into byte t%4 of the result, the others as they are
            const uint32_t sel = (0x03020100u & ~(0xFFu << (8 * (t % 4)))) |
                                 (uint32_t)(4 + sl % 4) << (8 * (t % 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t w = sl < 8 ? (sl < 4 ? cur[k][0] : cur[k][1]) : (sl < 12 ? cur[k][2] : cur[k][3]);
                out[k][t / 4] = __builtin_amdgcn_perm(w, out[k][t / 4], sel);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!plain) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float v[4];
                    decode4(out[k][w], v);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = e == 255 ? 0.0f : __builtin_amdgcn_ldexpf(v[j], __builtin_amdgcn_readlane(by, 4 * w + j));
                    out[k][w] = encode4(v[0], v[1], v[2], v[3]);
                }
            }
            *(u32x4_t *)(all + (blk * D + pair * 2 + k) * kKvBlock) = out[k];
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
    const int64_t jobs = (2 * (int64_t)a.c.heads + 3) / 4;
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
