// mq_attn_cached.hip -- attention of a few new tokens over the 8-bit key/value cache.
//
// out = softmax(scale q K^T) V over one pass of the cache: each wave holds a running maximum m,
// a running sum l and the unnormalised output O of 16 query rows (the query heads of one
// key/value head times the new tokens) and takes 64 cached tokens at a time:
//   S^T = K Q^T            v_mfma 16x16x32, the codes decoded exactly to dtype
//   P   = 2^(S - m)        in fp32, on the accumulator registers
//   O^T += V^T P^T         v_mfma 16x16x32 in bf16, P in two parts
// The products are laid out so that no value changes lanes between them. In step t of the first
// product, row m of the tile is token 4t + m%4 of the tile's block m/4; its result then leaves
// lane group g = lane/16 with tokens 4t..4t+3 of block g, and after four steps with all 16
// tokens of one block: the operand that the second product wants from that group, under one
// scale of K and one of V. The cache keeps a block's values token by token within a dimension,
// so the other operand is a 16-byte load.
//
// Bound by the bytes of the cache, read once: 131071 tokens, 32 query heads on 8 of 128, are 269 MB
// in 51 to 53 us, 5.1 to 5.3 TB/s (reads of 8 KB pieces in any order reach 5.8 on this card; the
// whole call takes 56 to 58 us). 32 sequences of up to 4096 tokens, 107 MB, take 31 us: each unit
// is one workgroup here, of 64 tiles at most and 26 in the mean, at 0.4 us each.
#include "mq_attn_device.hpp"

#include <cfloat>

namespace mq {
namespace {

constexpr int kTile = 64; // tokens a wave takes at a time: one block for each lane group
constexpr int kRows = 16; // query rows of a workgroup
constexpr int kWaves = 4;
constexpr int kCus = 256;
constexpr float kUnseen = -FLT_MAX; // in the kept scores: a token that the row does not see

// Work is cut along the cache into pieces, a workgroup to each. With `per` the whole call's tiles
// shared out to as many workgroups as the chip holds at a time, a unit (the kRows query rows of
// one sequence and key/value head) has as many equal pieces as tiles / per rounds to, one at
// least, in whole rounds of the waves (rounded up instead: 32 sequences of 1000 to 2000 tokens,
// 16 heads on 4 of 256, 36 us in place of 28; others within 6% either way). There are then at
// most units + groups pieces, which the host can launch without the lengths; each workgroup finds
// its piece by prefix sums over the sequences, and those past the last leave at once. A unit of
// several pieces is joined by a second launch.
//
// Without pieces, a workgroup takes a whole unit and there is no second launch (3 us and more).
// That is done where no sequence has more than 16 tiles, or at most 64 and there is a unit for
// every CU: then the units keep the chip busy by themselves unless a few of them hold most of the
// tokens, which the host does not know. Whole against cut, 32 query heads on 8 of 128: 1 x 1000
// tokens 9.4 and 10.7 us, 1 x 2000 14.9 and 10.8; 16 sequences (128 units) of 1 to 4000 tokens 26.5
// and 21.2; 32 (256 units) of 1 to 2000 17.1 and 23.1, of 1 to 4000 28.6 and 32.8; 64 of 2000 to
// 4000 75 and 79; against it, one of 4000 among 500s 26.8 and 16.3. Above 64 tiles either can be
// right (32 of 8000 each 90 and 96, of 500 to 8000 evenly 57 and 62, but mostly short ones up to 8000
// 51 and 41, 64 of those 96 and 84), and cutting loses less where it is wrong.
struct CachedPlan {
    int rows, row_tiles; // query rows of a key/value head, in tiles of kRows
    int groups;          // workgroups that share the tiles; 0: one for each unit
    int slots;           // max_len up to whole tiles
    size_t ml, part, scores, bytes; // workspace offsets
};

constexpr int kTilesWhole = 16, kTilesOrCut = 64; // tiles of a sequence, in the rule above

// Workgroups that fit the 256 CUs together (by registers: 3, 2 or 1 to a CU). Tiles shared out to
// half or twice as many, heads of 128: 1 x 131071 tokens 46.0 and 48.5 us against 46.9 (from the
// last-level cache); 16 sequences of 1 to 4000 tokens 24 and 24 against 21.
constexpr int resident(int d) { return kCus * (d <= 64 ? 3 : (d <= 128 ? 2 : 1)); }

void place_workspace(CachedPlan &p, int64_t units, int d, bool weights)
{
    const size_t parts = (size_t)units + p.groups;
    p.ml = 0;
    p.part = p.ml + (p.groups || weights ? parts * kRows * 8 : 0);
    p.scores = p.part + (p.groups ? parts * kRows * d * 4 : 0);
    p.bytes = p.scores + (weights ? (size_t)units * kRows * p.slots * 4 : 0);
}

CachedPlan cached_plan(int n, int q_heads, int kv_heads, int d, int q_len, int max_len, bool weights)
{
    CachedPlan p;
    p.rows = q_heads / kv_heads * q_len;
    p.row_tiles = (p.rows + kRows - 1) / kRows;
    const int64_t units = (int64_t)n * kv_heads * p.row_tiles;
    const int64_t tiles = ((int64_t)max_len + kTile - 1) / kTile;
    p.groups = tiles <= kTilesWhole || (tiles <= kTilesOrCut && units >= kCus) ? 0 : resident(d);
    p.slots = (int)(tiles * kTile);
    place_workspace(p, units, d, weights);
    return p;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__device__ __forceinline__ int held_tokens(const CachedArgs &a, int s)
{
    const int64_t cap = (int64_t)a.max_pages * a.c.page;
    const int c = cap < a.max_len ? (int)cap : a.max_len;
    return clampi(a.lens[s], 0, c);
}

// The softmax's scale times a block's scale, 2^(e-127); NaN for e = 255.
__device__ __forceinline__ float block_scale(float s, int e)
{
    return e == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(s, e - 127);
}

__device__ __forceinline__ int tiles_of(const CachedArgs &a, int s)
{
    return (held_tokens(a, s) + kTile - 1) / kTile;
}

// A workgroup's share of `total` tiles of the sequences' units. Two rounds of the waves (cut()
// makes 8 tiles of a share of 6) in one workgroup to a CU are faster than one round in two: 1 x
// 16000 tokens 12.8 against 14.8 us, 8 of up to 8190 with weights 15.4 against 15.9. With fewer tiles
// than that, one round on as many CUs as it takes: 1 x 4000 tokens 11.1 against 12.0.
template <int D>
__device__ __forceinline__ int share(int total, const CachedArgs &a, const CachedPlan &pl)
{
    const int tiles = total * a.c.heads * pl.row_tiles;
    const int per = (tiles + resident(D) - 1) / resident(D), cu = (tiles + kCus - 1) / kCus;
    const int least = clampi(cu, kWaves, 6);
    return per < least ? least : per;
}

// Pieces of a unit of `tiles` tiles, of *size tiles each (the last one may have fewer).
__device__ __forceinline__ int cut(int tiles, int per, int *size)
{
    const int want = (int)((float)tiles * __builtin_amdgcn_rcpf((float)per) + 0.5f);
    const int count = want < 1 ? 1 : want;
    *size = ((tiles + count - 1) / count + kWaves - 1) / kWaves * kWaves;
    return tiles ? (tiles + *size - 1) / *size : 0;
}

// Sum of f(sequence) over sequences 0..s-1.
template <class F>
__device__ __forceinline__ int sum_before(int s, F f)
{
    int sum = 0;
    for (int base = 0; base < s; base += 64) {
        const int q = base + (threadIdx.x & 63);
        sum += __builtin_amdgcn_readlane(wave_prefix(q < s ? f(q) : 0), 63);
    }
    return sum;
}

// What a row's result is multiplied by. The sum is 0 only where the row saw no token (maximum -inf,
// result 0), or where all its scores are -inf (the maximum is then the lowest number: NaN).
__device__ __forceinline__ float inverse(float sum, float top)
{
    if (sum != 0.0f) return 1.0f / sum;
    return top == -INFINITY ? 0.0f : __builtin_nanf("");
}

template <int DT, int D>
__global__ void __launch_bounds__(64 * kWaves, resident(D) / kCus) attn_cached_kernel(CachedArgs a, CachedPlan pl)
{
    typedef typename Elem<DT>::x8 x8;
    constexpr int KS = D / 32;         // steps of 32 dimensions in the first product
    constexpr bool WIDE = D % 64 == 0; // 16-byte loads of K: two steps each
    constexpr int VT = D / 16;         // tiles of 16 dimensions in the second product
    constexpr int LD = D + 4;          // a row of the waves' results in LDS, in floats
    __shared__ __align__(16) float part_o[kWaves * kRows * LD];
    __shared__ float part_m[kWaves][kRows], part_l[kWaves][kRows];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    const int per_unit = a.c.heads * pl.row_tiles; // units of a sequence
    const int group = a.q_heads / a.c.heads;
    const int blocks = a.c.page / kKvBlock;

    int s, sub, len, begin, end; // the piece: tokens begin..end-1 of unit `sub` of sequence s
    if (pl.groups) {
        const int held = lane < a.n ? held_tokens(a, lane) : 0; // of the first 64 sequences
        const int held_tiles = (held + kTile - 1) / kTile;
        int total = __builtin_amdgcn_readlane(wave_prefix(held_tiles), 63);
        if (a.n > 64) total = sum_before(a.n, [&](int q) { return tiles_of(a, q); });
        const int per = share<D>(total, a, pl);
        // pieces of one unit of each sequence, before this workgroup's (in whole sequences at
        // most this many)
        const int at = blockIdx.x / per_unit;
        int index, pieces, size;
        if (a.n <= 64) {
            const int own = cut(held_tiles, per, &size), incl = wave_prefix(own);
            const uint64_t after = __ballot(incl > at);
            if (!after) return;
            s = __builtin_ctzll(after);
            len = __builtin_amdgcn_readlane(held, s);
            pieces = __builtin_amdgcn_readlane(own, s);
            size = __builtin_amdgcn_readlane(size, s);
            index = at - (__builtin_amdgcn_readlane(incl, s) - pieces);
        } else {
            if (!locate_unit(at, a.n, [&](int q) { return cut(tiles_of(a, q), per, &size); }, &s, &index))
                return;
            len = __builtin_amdgcn_readfirstlane(held_tokens(a, s));
            pieces = cut((len + kTile - 1) / kTile, per, &size);
        }
        index = index * per_unit + blockIdx.x % per_unit; // among the sequence's pieces
        sub = index / pieces;
        begin = index % pieces * size * kTile;
        end = begin + size * kTile < len ? begin + size * kTile : len;
    } else {
        s = blockIdx.x / per_unit;
        sub = blockIdx.x % per_unit;
        len = __builtin_amdgcn_readfirstlane(held_tokens(a, s));
        begin = 0;
        end = len;
    }

    const int h = sub / pl.row_tiles;
    // A tile's loads are issued as soon as the registers of the tile before are free: K's after
    // the first product, V's after the second. The page numbers come through the scalar cache,
    // so that waiting for them waits for no vector load.
    constexpr int STEP = kWaves * kTile;
    u32x2_t k[4][KS];
    u32x4_t v[VT];
    int ke, ve;
    struct Blocks {
        int b0, b1, b2, b3;
    };
    // blocks (of the cache) of the four 16-token parts of a tile, -1 where there is none
    const auto tile_blocks = [&](int t) {
        typedef const int32_t __attribute__((address_space(4))) *scalar_t;
        const scalar_t table = (scalar_t)(uintptr_t)(a.table + (int64_t)s * a.max_pages);
        int at[4], pi[4], page[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at[i] = t + i * kKvBlock < end ? t + i * kKvBlock : end - 1;
            pi[i] = page_of(a.c, at[i]);
            page[i] = table[pi[i]];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = (page[i] * a.c.heads + h) * blocks + slot_of(a.c, at[i], pi[i]) / kKvBlock;
            const bool live = ((uint32_t)page[i] < (uint32_t)a.c.pages) & (t + i * kKvBlock < end);
            b[i] = live ? b[i] : -1;
        }
        return Blocks{b[0], b[1], b[2], b[3]};
    };
    const auto pick = [](const Blocks &r, int i) {
        const int lo = i & 1 ? r.b1 : r.b0, hi = i & 1 ? r.b3 : r.b2;
        return i & 2 ? hi : lo;
    };
    // K rows 4t + n%4 of block n/4, and the scales of block g. What is no block is read as
    // block 0 and masked where it is used.
    const auto load_k = [&](int kb, int vb) {
        const uint8_t *p = a.c.kc + (int64_t)(kb < 0 ? 0 : kb) * (kKvBlock * D) + (n & 3) * D + g * (WIDE ? 16 : 8);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int i = 0; i < KS; i += WIDE ? 2 : 1) {
                if constexpr (WIDE) {
                    const u32x4_t w = *(const u32x4_t *)(p + t * 4 * D + i * 32);
                    k[t][i] = u32x2_t{w[0], w[1]};
                    k[t][i + 1] = u32x2_t{w[2], w[3]};
                } else {
                    k[t][i] = *(const u32x2_t *)(p + t * 4 * D + i * 32);
                }
            }
        ke = a.c.ks[vb < 0 ? 0 : vb];
        ve = a.c.vs[vb < 0 ? 0 : vb];
    };
    const auto load_v = [&](int vb) {
        const uint8_t *p = a.c.vc + (int64_t)(vb < 0 ? 0 : vb) * (kKvBlock * D) + n * kKvBlock;
#pragma unroll
        for (int i = 0; i < VT; ++i) v[i] = *(const u32x4_t *)(p + i * 16 * kKvBlock);
    };
    const int tv = g * kKvBlock; // the lane's block of a tile
    int vb = -1;
    const bool whole = begin == 0 && end == len;
    const int row = sub % pl.row_tiles * kRows + n;
    const int qi = row / group, qh = h * group + row % group;
    const bool real = row < pl.rows;
    // tokens this lane's row sees
    const int see = real ? clampi(len - a.q_len + qi + 1, 0, len) : 0;

    // the row's query, in the order in which the lanes hold K
    x8 q[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int d = WIDE ? i / 2 * 64 + g * 16 + i % 2 * 8 : i * 32 + g * 8;
        u32x4_t v = {0, 0, 0, 0};
        if (real) v = *(const u32x4_t *)(a.q.p + (int64_t)(s * a.q_len + qi) * a.q.ts + qh * a.q.hs + d);
        q[i] = __builtin_bit_cast(x8, v);
    }

    // The query is waited for here: left to its first use, inside the loop, the wait would empty
    // the queue of loads in every step.
    __builtin_amdgcn_s_waitcnt(0x0F70); // vmcnt(0)
    f32x4_t o[VT];
#pragma unroll
    for (int i = 0; i < VT; ++i) o[i] = f32x4_t{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    int t0 = begin + wave * kTile;
    if (t0 < end) {
        const Blocks r = tile_blocks(t0);
        vb = pick(r, g);
        load_k(pick(r, n >> 2), vb);
        load_v(vb);
    }
    for (; t0 < end; t0 += STEP) {
        Blocks r = {-1, -1, -1, -1};
        if (t0 + STEP < end) r = tile_blocks(t0 + STEP);

        // tokens of this lane's block that its row sees (0 where there is no block)
        const int sees = vb >= 0 ? see - (t0 + tv) : 0;
        const float kf = block_scale(a.scale_log2e, ke), vf = block_scale(1.0f, ve);
        float sc[16];
        float top = sees > 0 ? -FLT_MAX : -INFINITY; // -inf: a row that has seen nothing yet
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            f32x4_t acc = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < KS; ++i)
                acc = Elem<DT>::mfma16(decode8<DT>(k[t][i][0], k[t][i][1]), q[i], acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                sc[4 * t + r] = 4 * t + r < sees ? acc[r] * kf : -INFINITY;
                top = fmaxf(top, sc[4 * t + r]);
            }
        }
        // slots past the last token, and pages that do not exist, hold anything
        const bool ragged = t0 + kTile > end || __any(vb < 0);
        const int slots = vb >= 0 ? end - (t0 + tv) : 0;
        // Loaded also where there is no next tile (block 0 stands in): a load under a condition
        // would be copied, and so waited for, where the paths meet.
        vb = pick(r, g);
        load_k(pick(r, n >> 2), vb);

        if (a.weights && real) {
            float *dst = (float *)((char *)a.ws + pl.scores) +
                         ((int64_t)(s * per_unit + sub) * kRows + n) * pl.slots + t0 + tv;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                *(f32x4_t *)(dst + 4 * t) = f32x4_t{4 * t < sees ? sc[4 * t] : kUnseen, 4 * t + 1 < sees ? sc[4 * t + 1] : kUnseen,
                                                    4 * t + 2 < sees ? sc[4 * t + 2] : kUnseen, 4 * t + 3 < sees ? sc[4 * t + 3] : kUnseen};
        }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float base = m_new == -INFINITY ? 0.0f : m_new;
        if (__any(m_new > m)) { // some row's maximum grew
            const float keep = __builtin_amdgcn_exp2f(m - base);
            l *= keep;
#pragma unroll
            for (int i = 0; i < VT; ++i) o[i] *= keep;
        }
        m = m_new;
        float p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float e = __builtin_amdgcn_exp2f(sc[j] - base);
            l += e;
            p[j] = j < sees ? e * vf : 0.0f; // a masked place adds nothing, whatever lies there
        }
        if (ragged) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int b = clampi(slots - 4 * w, 0, 4);
                const uint32_t mask = b == 4 ? ~0u : (1u << (8 * b)) - 1u;
#pragma unroll
                for (int i = 0; i < VT; ++i) v[i][w] &= mask;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            u32x4_t ph, pr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a0 = p[8 * u + 2 * j], a1 = p[8 * u + 2 * j + 1];
                ph[j] = Elem<MQ_BF16>::pack(a0, a1);
                // bf16 has the range of p times a block's scale and holds it to 2^-8; what that leaves
                // goes in as a second part, and both hold it to 2^-16, so that the output's own
                // rounding is the one that counts. The second product is not what bounds the kernel:
                // 32 sequences up to 4096 tokens 26.6 us with one part and 27.8 with both, others
                // within 2%.
                pr[j] = Elem<MQ_BF16>::pack(a0 - __uint_as_float(ph[j] << 16),
                                            a1 - __uint_as_float(ph[j] & 0xFFFF0000u));
            }
            const bf16x8_t hi = __builtin_bit_cast(bf16x8_t, ph), lo = __builtin_bit_cast(bf16x8_t, pr);
#pragma unroll
            for (int i = 0; i < VT; ++i) {
                const bf16x8_t vv = decode8<MQ_BF16>(v[i][2 * u], v[i][2 * u + 1]);
                o[i] = Elem<MQ_BF16>::mfma16(vv, hi, o[i]);
                o[i] = Elem<MQ_BF16>::mfma16(vv, lo, o[i]);
            }
        }
        load_v(vb);
    }
    // the four lane groups hold parts of l, the waves parts of everything
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        part_m[wave][n] = m;
        part_l[wave][n] = l;
    }
    if (real) {
#pragma unroll
        for (int i = 0; i < VT; ++i)
            *(f32x4_t *)&part_o[(wave * kRows + n) * LD + i * 16 + g * 4] = o[i];
    }
    __syncthreads();
    float top = part_m[0][n];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, part_m[w][n]);
    const float base = top == -INFINITY ? 0.0f : top;
    float f[kWaves], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        f[w] = __builtin_amdgcn_exp2f(part_m[w][n] - base);
        sum += part_l[w][n] * f[w];
    }
    const float inv = inverse(sum, top);
    const int64_t slot = blockIdx.x;
    if ((!whole || a.weights) && wave == 0 && g == 0)
        ((f32x2_t *)((char *)a.ws + pl.ml))[slot * kRows + n] = f32x2_t{top, sum};
    if (real) {
        uint16_t *out = a.out + (int64_t)(s * a.q_len + qi) * a.out_ts + qh * a.out_hs;
        float *part = (float *)((char *)a.ws + pl.part) + (slot * kRows + n) * D;
#pragma unroll
        for (int j = 0; j < (VT + kWaves - 1) / kWaves; ++j) { // each wave finishes some dimensions
            const int i = j * kWaves + wave;
            if (i >= VT) break;
            f32x4_t v = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                v += *(const f32x4_t *)&part_o[(w * kRows + n) * LD + i * 16 + g * 4] * f[w];
            if (whole)
                *(u32x2_t *)(out + i * 16 + g * 4) = u32x2_t{Elem<DT>::pack(v[0] * inv, v[1] * inv),
                                                             Elem<DT>::pack(v[2] * inv, v[3] * inv)};
            else
                *(f32x4_t *)(part + i * 16 + g * 4) = v;
        }
    }
}

// What is left once every part is done, in one launch: the first workgroups join the parts of a
// query row along the cache (kJoinThreads / (D/4) parts at a time, four dimensions to a lane),
// the others add the weights of 256 tokens, summed over the rows in order, to their places. Bound
// by the latency of the launch and of three loads that wait for each other (lengths, maxima and
// sums, parts): 5.5 us at 131071 tokens, 8 us with the weights of 8 of up to 8190.
constexpr int kJoinThreads = 256;

template <int DT, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(CachedArgs a, CachedPlan pl, int join)
{
    constexpr int Q = D / 4, G = kJoinThreads / Q; // lanes of a part, parts at a time
    __shared__ __align__(16) float acc[G][D];
    __shared__ f32x2_t row_ml[kRows];
    __shared__ uint64_t sharing[kJoinThreads / 64]; // 64 sequences, a bit to each
    const int tid = threadIdx.x;
    const int group = a.q_heads / a.c.heads;
    const f32x2_t *ml = (const f32x2_t *)((const char *)a.ws + pl.ml);

    const int per_unit = a.c.heads * pl.row_tiles;
    // what this workgroup works on
    const bool adds = (int)blockIdx.x >= join; // weights
    const int chunks = (pl.slots + kJoinThreads - 1) / kJoinThreads;
    const int sh = adds ? ((int)blockIdx.x - join) / chunks : (int)blockIdx.x / pl.rows;
    const int s = sh / a.c.heads, h = sh % a.c.heads;
    // tokens of a sequence, the pieces of one unit of it and of those before
    struct Seq {
        int len, pieces, before;
    };
    int held = 0, own = 0, incl = 0, per = 0; // lane q: sequence q, where there are 64 or fewer
    if (pl.groups && a.n > 64) {
        per = share<D>(sum_before(a.n, [&](int q) { return tiles_of(a, q); }), a, pl);
    } else if (pl.groups) { // one load
        const int lane = tid & 63;
        held = lane < a.n ? held_tokens(a, lane) : 0;
        const int tiles = (held + kTile - 1) / kTile;
        int size;
        per = share<D>(__builtin_amdgcn_readlane(wave_prefix(tiles), 63), a, pl);
        own = cut(tiles, per, &size);
        incl = wave_prefix(own);
    }
    const auto sequence = [&](int q) {
        if (!pl.groups) return Seq{held_tokens(a, q), 1, q};
        if (a.n <= 64) {
            const int pieces = __builtin_amdgcn_readlane(own, q);
            return Seq{__builtin_amdgcn_readlane(held, q), pieces, __builtin_amdgcn_readlane(incl, q) - pieces};
        }
        int size;
        const auto pieces_of = [&](int x) { return cut(tiles_of(a, x), per, &size); };
        return Seq{held_tokens(a, q), pieces_of(q), sum_before(q, pieces_of)};
    };
    const Seq seq = sequence(s);
    const int pieces = seq.pieces;

    if (adds) {
        const int first = ((int)blockIdx.x - join) % chunks * kJoinThreads, t = first + tid;
        if (first >= seq.len) return;
        // The weight of token t that sequence q's rows give it, by the whole workgroup.
        const auto given = [&](int q, const Seq &x) {
            float sum = 0.0f;
            for (int rt = 0; rt < pl.row_tiles; ++rt) {
                // maximum and sum of the tile's rows: 16 lanes a row, each every 16th part
                const int r = tid / 16;
                const int rows = pl.rows - rt * kRows < kRows ? pl.rows - rt * kRows : kRows;
                const float *sc = (const float *)((const char *)a.ws + pl.scores) +
                                  ((int64_t)(q * a.c.heads + h) * pl.row_tiles + rt) * kRows * pl.slots +
                                  (t < x.len ? t : 0);
                float score[kRows]; // on their way while the maxima are found
#pragma unroll
                for (int i = 0; i < kRows; ++i) score[i] = sc[(int64_t)(i < rows ? i : 0) * pl.slots];
                const int64_t slot = (int64_t)x.before * per_unit + (h * pl.row_tiles + rt) * x.pieces;
                const f32x2_t *p = ml + slot * kRows + r;
                float top = -INFINITY, l = 0.0f;
                for (int i = tid % 16; i < x.pieces; i += 16) top = fmaxf(top, p[(int64_t)i * kRows][0]);
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
                const float base = top == -INFINITY ? 0.0f : top;
                for (int i = tid % 16; i < x.pieces; i += 16) {
                    const f32x2_t v = p[(int64_t)i * kRows];
                    l += v[1] * __builtin_amdgcn_exp2f(v[0] - base);
                }
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) l += __shfl_xor(l, d);
                __syncthreads();
                if (tid % 16 == 0) row_ml[r] = f32x2_t{base, inverse(l, top)};
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    if (i >= rows) continue;
                    const float p = __builtin_amdgcn_exp2f(score[i] - row_ml[i][0]) * row_ml[i][1];
                    // nothing from a row that does not see the token: the row may be NaN
                    sum += score[i] != kUnseen ? p : 0.0f;
                }
            }
            return sum;
        };
        // Sequences may have pages in common (the beginning of a prompt). The first of those that
        // hold a token in such a page adds the weights of all of them, one after another, so the
        // order of the sum is fixed. They are looked for at the same place of their tables, a wave's
        // pages against 64 sequences at a time. Where there are none, looking takes 1.3 us of 19 (8
        // sequences up to 8190 tokens, 4 heads) and 6 us of 40 (128 up to 2000).
        const auto page_at = [&](int q, int column) { return a.table[(int64_t)q * a.max_pages + column]; };
        constexpr int W = kJoinThreads / 64, C = kJoinThreads / kKvBlock / W; // pages to a wave, at most
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int last = (first + kJoinThreads < seq.len ? first + kJoinThreads : seq.len) - 1;
        const int c0 = page_of(a.c, first), c1 = page_of(a.c, last);
        const int holds = lane < a.n ? held_tokens(a, lane) : 0;
        int there[C], ours[C], from[C]; // of the wave's pages; the tokens before each
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = c0 + wave + i * W;
            there[i] = ours[i] = -1;
            from[i] = INT32_MAX;
            if (c > c1) continue;
            from[i] = c * a.c.page;
            there[i] = page_at(lane < a.n ? lane : s, c);
            ours[i] = page_at(s, c);
        }
        const int pi = page_of(a.c, t < last ? t : last), page = page_at(s, pi);
        bool mine = t <= last && page >= 0 && page < a.c.pages;
        float sum = given(s, seq);
        bool common = false;
#pragma unroll
        for (int i = 0; i < C; ++i) common |= lane != s && holds > from[i] && there[i] == ours[i];
        for (int q = lane + 64; q < a.n; q += 64) {
            const int has = held_tokens(a, q);
#pragma unroll
            for (int i = 0; i < C; ++i)
                if (c0 + wave + i * W <= c1)
                    common |= q != s && has > from[i] && page_at(q, c0 + wave + i * W) == ours[i];
        }
        if (__syncthreads_or(common)) {
            for (int q0 = 0; q0 < a.n; q0 += 64) {
                const int q = q0 + lane, has = q < a.n ? held_tokens(a, q) : 0;
                uint64_t m = 0; // of these 64, those with one of the wave's pages
                for (int i = 0; i < C; ++i)
                    m |= __ballot(has > from[i] && q != s && page_at(q, c0 + wave + i * W) == ours[i]);
                __syncthreads(); // the last 64 have been read
                if (lane == 0) sharing[wave] = m;
                __syncthreads();
                m = sharing[0];
#pragma unroll
                for (int w = 1; w < W; ++w) m |= sharing[w];
                for (; m; m &= m - 1) {
                    const int other = __builtin_amdgcn_readfirstlane(q0 + __builtin_ctzll(m));
                    const bool too = t < held_tokens(a, other) && page_at(other, pi) == page;
                    if (other < s) { // it adds them, if it holds the token too
                        mine &= !too;
                        continue;
                    }
                    if (!__syncthreads_or(mine)) return;
                    const float more = given(other, sequence(other));
                    if (too) sum += more;
                }
            }
        }
        // A page that two rows have at different places is no such case, nor one that is twice in a
        // row; the additions to it are atomic, in any order.
        if (mine) unsafeAtomicAdd(a.weights + ((int64_t)page * a.c.heads + h) * a.c.page + slot_of(a.c, t, pi), sum);
        return;
    }

    const int r0 = blockIdx.x % pl.rows;
    const int qi = r0 / group, qh = h * group + r0 % group;
    const int sub = h * pl.row_tiles + r0 / kRows;
    if (pieces == 1) return; // written by its only workgroup
    const int64_t slot = (int64_t)seq.before * per_unit + sub * pieces;
    ml += slot * kRows + r0 % kRows;
    const float *po = (const float *)((const char *)a.ws + pl.part) + (slot * kRows + r0 % kRows) * D;
    const int lane = tid & 63;
    // every wave finds the row's maximum and sum for itself
    float top = -INFINITY, l = 0.0f;
    for (int i = lane; i < pieces; i += 64) top = fmaxf(top, ml[(int64_t)i * kRows][0]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float base = top == -INFINITY ? 0.0f : top;
    for (int i = lane; i < pieces; i += 64) {
        const f32x2_t v = ml[(int64_t)i * kRows];
        l += v[1] * __builtin_amdgcn_exp2f(v[0] - base);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
    const float inv = inverse(l, top);
    const int g = tid / Q, c = tid % Q;
    if (g < G) {
        f32x4_t o = {0, 0, 0, 0};
#pragma unroll 4
        for (int i = g; i < pieces; i += G)
            o += *(const f32x4_t *)(po + (int64_t)i * kRows * D + c * 4) *
                 __builtin_amdgcn_exp2f(ml[(int64_t)i * kRows][0] - base);
        *(f32x4_t *)&acc[g][c * 4] = o;
    }
    __syncthreads();
    if (tid >= Q) return;
    f32x4_t o = {0, 0, 0, 0};
    for (int i = 0; i < G && i < pieces; ++i) o += *(const f32x4_t *)&acc[i][tid * 4];
    uint16_t *dst = a.out + (int64_t)(s * a.q_len + qi) * a.out_ts + qh * a.out_hs + tid * 4;
    *(u32x2_t *)dst = u32x2_t{Elem<DT>::pack(o[0] * inv, o[1] * inv), Elem<DT>::pack(o[2] * inv, o[3] * inv)};
}

template <int DT, int D>
hipError_t cached(const CachedArgs &a, hipStream_t st)
{
    const CachedPlan pl = cached_plan(a.n, a.q_heads, a.c.heads, D, a.q_len, a.max_len, a.weights != nullptr);
    const int64_t units = (int64_t)a.n * a.c.heads * pl.row_tiles;
    // tiles, and the pieces of all units, are counted in 32 bits
    if (units * (pl.slots / kTile + 1) + resident(D) > INT32_MAX) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(units + pl.groups);
    attn_cached_kernel<DT, D><<<grid, 64 * kWaves, 0, st>>>(a, pl);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t join = pl.groups ? (int64_t)a.n * a.c.heads * pl.rows : 0;
    const int64_t add = a.weights ? (int64_t)a.n * a.c.heads * ((pl.slots + kJoinThreads - 1) / kJoinThreads) : 0;
    if (join + add > INT32_MAX) return hipErrorInvalidValue;
    if (join + add == 0) return hipSuccess;
    attn_join_kernel<DT, D><<<(unsigned)(join + add), kJoinThreads, 0, st>>>(a, pl, (int)join);
    return hipGetLastError();
}

template <int DT>
hipError_t cached_dim(const CachedArgs &a, int d, hipStream_t st)
{
    switch (d) {
    case 64: return cached<DT, 64>(a, st);
    case 96: return cached<DT, 96>(a, st);
    case 128: return cached<DT, 128>(a, st);
    case 192: return cached<DT, 192>(a, st);
    case 256: return cached<DT, 256>(a, st);
    }
    return hipErrorInvalidValue;
}

} // namespace

size_t attn_cached_workspace(int n, int q_heads, int kv_heads, int d, int q_len, int max_len,
                             bool weights)
{
    CachedPlan p = cached_plan(n, q_heads, kv_heads, d, q_len, max_len, weights);
    const size_t bytes = p.bytes;
    if (p.groups || p.slots <= kTilesWhole * kTile) return bytes;
    // enough for a call with fewer sequences too, whose units are cut
    p.groups = resident(d);
    place_workspace(p, kCus - 1, d, weights);
    return bytes > p.bytes ? bytes : p.bytes;
}

hipError_t launch_attn_cached(const CachedArgs &a, int d, int dtype, hipStream_t st)
{
    if (a.n == 0) return hipSuccess;
    return dtype == MQ_BF16 ? cached_dim<MQ_BF16>(a, d, st) : cached_dim<MQ_F16>(a, d, st);
}

} // namespace mq
