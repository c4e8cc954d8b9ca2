// mq_mx4_quantize.hip -- microscaled 4-bit quantization along rows and columns, and back.
//
// A block of 32 gets the smallest power of two that brings its largest magnitude to 6 or less, as a
// byte, and 32 codes of 4 bits. Every kernel reads its input once: where rows and columns are wanted,
// a wave holds a tile of 64 columns in registers and takes the blocks of both directions from them.
//
// Bound by memory: 8192 x 4096 along both directions 22 us from bf16 (103 MB, 4.6 TB/s) and 39 from fp32
// (170 MB, 4.4), rows alone 14.7 (85 MB, 5.8); gradients of 4096 x 8192 65 us (272 MB, 4.2 TB/s). Small ones by a
// wave's own length: 500 x 1000 3.9 us with 4 rows to a lane, 8.5 with 32. Stochastic rounding (a Philox call
// to 8 elements and direction) takes 8192 x 4096 bf16 to 45 us.
#include "mq_mx4_device.hpp"

namespace mq {
namespace {

constexpr int64_t kMaxGroups = UINT32_MAX / 256; // a grid's threads are counted in 32 bits

// Where row r of piece p lies, in rows of pieces.
__device__ __forceinline__ int64_t place(const Mx4View &q, int p, int64_t r) { return (int64_t)p * q.rows + r; }

// ---- rows alone ---------------------------------------------------------------------------------
//
// 8 columns and U rows to a thread, 4 threads to a block.
template <int DT, bool SR, int U, bool TAIL>
__global__ void __launch_bounds__(256) mx4_quantize_rows_kernel(Mx4QuantArgs a, int width, int across)
{
    typedef typename Dense<DT>::T T;
    const int groups = a.row.pieces() * 32;
    const int g = (int)(blockIdx.x % across) * width + (int)(threadIdx.x % width);
    const int r0 = (int)(blockIdx.x / across * (256 / width) + threadIdx.x / width) * U; // below 2^30 + 1024
    if (g >= groups) return; // whole quads: groups is a multiple of 32
    if (r0 >= a.rows) return;
    const Reach reach = reach_of(g * 8, a.cols);
    Eight<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = load8<TAIL>(static_cast<const T *>(a.x.p) + (int64_t)min(r0 + u, a.rows - 1) * a.x.stride, reach, a.cols);
    const int blocks = (a.cols + 31) / 32;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (r0 + u >= a.rows) return;
        float v[8];
        values8<DT, TAIL>(raw[u], reach, v);
        const uint32_t e = mx4_scale(quad_max(amax8(v)));
        const uint64_t n = 4 * ((uint64_t)(r0 + u) * blocks) + g;
        const int64_t at = place(a.row, g >> 5, r0 + u);
        *(uint32_t *)(a.row.codes + at * 128 + (g & 31) * 4) = encode8<SR>(v, e, n, 0, a.seed_lo, a.seed_hi);
        if ((g & 3) == 0) a.row.scales[at * 8 + (g & 31) / 4] = (uint8_t)e;
    }
}

// ---- rows and columns -----------------------------------------------------------------------------
//
// Lane (q, cg) of a wave holds NR rows of 8 columns: 8 NR rows of 64 columns to a wave, and four waves
// beside each other, so that rows are read in long runs (one above another: gradients of 4096 x 8192
// 80 us in place of 61). A row's block lies in a quad of lanes; a column's in
// 32 / NR lanes, 8 lanes apart (NR = 4 or 8; 32 rows of 16-bit elements: the kernel behind this one).

// Eight values to quantize: of x, or of dg and du of h = silu(g) u.
template <int DT, bool GRAD, bool TAIL, bool PASS> struct Source {
    static constexpr int K = GRAD ? 2 : 1;
    static __device__ __forceinline__ void load(const Mx4QuantArgs &a, int64_t r, Reach at, float (*v)[8])
    {
        typedef typename Dense<DT>::T T;
        const auto get = [&](const MatView &m, float *to) {
            values8<DT, TAIL>(load8<TAIL, PASS>(static_cast<const T *>(m.p) + r * m.stride, at, a.cols), at, to);
        };
        get(a.x, v[0]);
        if constexpr (GRAD) {
            float g[8], u[8];
            get(a.g, g);
            get(a.u, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dh = v[0][i], s = sigmoid(g[i]), gs = g[i] * s;
                v[0][i] = dh * u[i] * __builtin_fmaf(gs, 1.0f - s, s); // s (1 + g (1 - s))
                v[1][i] = dh * gs;
            }
        }
    }
};

// Largest value of this lane and the one 16 (32) lanes away.
__device__ __forceinline__ uint32_t max_lane_xor_16(uint32_t v)
{
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max_u32(s[0], s[1]);
}
__device__ __forceinline__ uint32_t max_lane_xor_32(uint32_t v)
{
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max_u32(s[0], s[1]);
}

template <int DT, bool GRAD, int NR, bool SR, bool TAIL, bool PASS>
__global__ void __launch_bounds__(256, 2) mx4_quantize_both_kernel(Mx4QuantArgs a, int across)
{
    static_assert(NR == 4 || NR == 8, "a column's block is in four lanes or eight");
    constexpr int K = Source<DT, GRAD, TAIL, PASS>::K, WR = 8 * NR; // rows of a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 3, cg = lane & 7;
    const int c0 = ((int)(blockIdx.x % across) * 4 + wave) * 64, c = c0 + cg * 8;
    const int r0 = (int)(blockIdx.x / across) * WR + q * NR;
    if (c0 >= (a.row.codes ? a.row.pieces() * 256 : a.cols)) return;
    const Reach reach = reach_of(c, a.cols);
    float v[K][NR][8];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float t[K][8];
        Source<DT, GRAD, TAIL, PASS>::load(a, min(r0 + r, a.rows - 1), reach, t);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][r][i] = r0 + r < a.rows ? t[k][i] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Mx4View &row = k ? a.row2 : a.row, &col = k ? a.col2 : a.col;
        if (row.codes) {
            const int g = c / 8, blocks = (a.cols + 31) / 32;
            const int64_t at = place(row, g >> 5, r0);
            uint32_t *to = (uint32_t *)(row.codes + at * 128 + (g & 31) * 4);
            uint8_t *zs = row.scales + at * 8 + (g & 31) / 4;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const uint32_t e = mx4_scale(quad_max(amax8(v[k][r])));
                const uint64_t n = 4 * ((uint64_t)(r0 + r) * blocks) + g;
                const uint32_t codes = encode8<SR>(v[k][r], e, n, 2 * k, a.seed_lo, a.seed_hi);
                if (r0 + r >= a.rows) continue;
                to[r * 32] = codes;
                if ((g & 3) == 0) zs[r * 8] = (uint8_t)e;
            }
        }
        if (col.codes) {
            const int blocks = (a.rows + 31) / 32, part = r0 & 255; // first row within the piece
            const int64_t at = place(col, r0 >> 8, c);
            uint8_t *const first = col.codes + at * 128 + (part & ~7) / 2, *const zs = col.scales + at * 8 + part / 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t amax = 0;
#pragma unroll
                for (int r = 0; r < NR; ++r) amax = max_u32(amax, __float_as_uint(v[k][r][i]) & 0x7FFFFFFFu);
                amax = max_u32(amax, (uint32_t)__builtin_amdgcn_mov_dpp((int)amax, 0x128, 0xF, 0xF, true)); // lane ^ 8
                amax = max_lane_xor_16(amax);
                if constexpr (NR < 8) amax = max_lane_xor_32(amax);
                const uint32_t e = mx4_scale(amax);
                if (c + i >= a.cols) continue;
                float t[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = v[k][j % NR][i]; // (NR = 4: twice, in either half's place)
                const uint64_t n = 4 * ((uint64_t)(c + i) * blocks) + (uint64_t)(r0 / 8);
                const uint32_t codes = encode8<SR>(t, e, n, 2 * k + 1, a.seed_lo, a.seed_hi);
                uint32_t *to = (uint32_t *)(first + i * 128);
                if constexpr (NR == 8) *to = codes;
                else ((uint16_t *)to)[part / 4 % 2] = (uint16_t)(part & 4 ? codes >> 16 : codes);
                if (part % 32 == 0) zs[i * 8] = (uint8_t)e;
            }
        }
    }
}

// The same for 16-bit elements rounded to nearest, two to a register all the way: NR = 32.
template <int DT, bool TAIL>
__global__ void __launch_bounds__(256, 2) mx4_quantize_packed_kernel(Mx4QuantArgs a, int across)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 3, cg = lane & 7;
    const int down = blockIdx.x / across;
    const int c0 = ((int)(blockIdx.x % across) * 4 + wave) * 64, c = c0 + cg * 8;
    const int r0 = down * 256 + q * 32;
    if (c0 >= (a.row.codes ? a.row.pieces() * 256 : a.cols)) return;
    const uint16_t *x = static_cast<const uint16_t *>(a.x.p) + (int64_t)r0 * a.x.stride;
    const Reach reach = reach_of(c, a.cols);
    Eight<uint16_t> raw[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) raw[r] = load8<TAIL, true>(x + (int64_t)min(r, a.rows - 1 - r0) * a.x.stride, reach, a.cols);
    u32x4_t d[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        d[r] = __builtin_bit_cast(u32x4_t, shifted<TAIL>(raw[r], reach));
        if (r0 + r >= a.rows) d[r] = u32x4_t{0, 0, 0, 0};
    }
    typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
    typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;
    const auto max2 = [](uint32_t m, uint32_t v) {
        const u16x2_t x = __builtin_bit_cast(u16x2_t, m), y = __builtin_bit_cast(u16x2_t, v & 0x7FFF7FFFu);
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(x, y));
    };
    const auto scale_of = [](uint32_t half) { return mx4_scale(__float_as_uint(Dense<DT>::load((uint16_t)half))); };
    const auto code2 = [](uint32_t c, uint32_t two, float by, auto at) {
        if constexpr (DT == MQ_BF16) return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, two), by, decltype(at)::value);
        else return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2_t, two), by, decltype(at)::value);
    };
    const auto codes8 = [&](uint32_t e, uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3) {
        const float by = __uint_as_float((e == 255 ? 127u : e) << 23);
        uint32_t k = code2(0, x0, by, Int<0>{});
        k = code2(k, x1, by, Int<1>{});
        k = code2(k, x2, by, Int<2>{});
        k = code2(k, x3, by, Int<3>{});
        return e == 255 ? 0u : k;
    };
    if (a.row.codes) {
        const int g = c / 8;
        const int64_t at0 = place(a.row, g >> 5, r0);
        uint32_t *to = (uint32_t *)(a.row.codes + at0 * 128 + (g & 31) * 4);
        uint8_t *zs = a.row.scales + at0 * 8 + (g & 31) / 4;
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            uint32_t m = max2(max2(max2(max2(0u, d[r][0]), d[r][1]), d[r][2]), d[r][3]);
            m = quad_max(max_u32(m & 0xFFFFu, m >> 16));
            const uint32_t e = scale_of(m), k = codes8(e, d[r][0], d[r][1], d[r][2], d[r][3]);
            if (r0 + r < a.rows) {
                to[r * 32] = k;
                if ((g & 3) == 0) zs[r * 8] = (uint8_t)e;
            }
        }
    }
    if (a.col.codes) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int r = 0; r < 32; ++r) m = max2(m, d[r][k]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t e = scale_of(half ? m >> 16 : m & 0xFFFFu);
                u32x4_t codes;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t two[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        two[j] = __builtin_amdgcn_perm(d[8 * w + 2 * j + 1][k], d[8 * w + 2 * j][k], half ? 0x07060302u : 0x05040100u);
                    codes[w] = codes8(e, two[0], two[1], two[2], two[3]);
                }
                const int i = c + 2 * k + half;
                if (i >= a.cols) continue;
                const int64_t at = place(a.col, down, i);
                *(u32x4_t *)(a.col.codes + at * 128 + q * 16) = codes;
                a.col.scales[at * 8 + q] = (uint8_t)e;
            }
        }
    }
}

// ---- back -----------------------------------------------------------------------------------------

// 8 columns to a thread.
template <int DT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(Mx4View q, MatView out, bool through, int width, int across)
{
    typedef typename Dense<DT>::T T;
    const int g = (int)(blockIdx.x % across) * width + (int)(threadIdx.x % width);
    const int64_t r = blockIdx.x / across * (int64_t)(256 / width) + threadIdx.x / width;
    if (g * 8 >= q.cols || r >= q.rows) return;
    const int64_t at = place(q, g >> 5, r);
    const uint32_t codes = *(const uint32_t *)(q.codes + at * 128 + (g & 31) * 4);
    const uint32_t e = q.scales[at * 8 + (g & 31) / 4];
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = codes >> (4 * j);
        const float m = elem_mag_to_float<kFP4>(c & 7u);
        const float x = __builtin_amdgcn_ldexpf(c & 8u ? -m : m, (int)e - 127);
        v[j] = Dense<DT>::store(e == 255 ? __uint_as_float(0x7FC00000u) : x);
    }
    T *to = static_cast<T *>(out.p) + r * out.stride + g * 8;
    if (g * 8 + 8 <= q.cols) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
            typedef u32x4_t Any __attribute__((aligned(2)));
            const u32x4_t w = ((const u32x4_t *)v)[j];
            if (sizeof(T) == 2 && through) store_past((u32x4_t *)to + j, w);
            else *(Any *)((u32x4_t *)to + j) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (g * 8 + j < q.cols) to[j] = v[j];
    }
}

// Threads to a row of `groups`, of a workgroup's 256.
int width_of(int groups)
{
    int w = 32;
    while (w < 256 && w < groups) w *= 2;
    return w;
}

template <int DT, bool SR>
hipError_t rows_alone(const Mx4QuantArgs &a, hipStream_t st)
{
    const int groups = a.row.pieces() * 32, width = width_of(groups), across = (groups + width - 1) / width;
    // four rows to a thread hide the loads' latency, where that leaves two workgroups for every CU: 1024 x 4096 bf16
    // 3.9 -> 3.4 us, 8192 x 4096 15.4 -> 14.7 (fp32, longer loads, 5.1 and 5.2, 29.6 and 31.2); 256 x 4096 2.7 and 2.9
    const bool four = (int64_t)across * a.rows * width >= 4 * 256 * 512;
    const int per = 256 / width * (four ? 4 : 1);
    const int64_t grid = ((int64_t)a.rows + per - 1) / per * across;
    if (grid > kMaxGroups) return hipErrorInvalidValue;
    const auto run = [&](auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        if (four) mx4_quantize_rows_kernel<DT, SR, 4, TAIL><<<(uint32_t)grid, 256, 0, st>>>(a, width, across);
        else mx4_quantize_rows_kernel<DT, SR, 1, TAIL><<<(uint32_t)grid, 256, 0, st>>>(a, width, across);
    };
    if (a.cols % 8) run(Int<1>{});
    else run(Int<0>{});
    return hipGetLastError();
}

template <int DT, bool GRAD, int NR, bool SR>
hipError_t both(const Mx4QuantArgs &a, hipStream_t st)
{
    const int cols = a.row.codes ? a.row.pieces() * 256 : a.cols, across = (cols + 255) / 256;
    const int64_t grid = ((int64_t)a.rows + 255) / 256 * (32 / NR) * across; // whole pieces of columns
    if (grid > kMaxGroups) return hipErrorInvalidValue;
    const auto run = [&](auto tail, auto pass) {
        constexpr bool TAIL = decltype(tail)::value, PASS = decltype(pass)::value;
        if constexpr (NR == 32) mx4_quantize_packed_kernel<DT, TAIL><<<(uint32_t)grid, 256, 0, st>>>(a, across);
        else mx4_quantize_both_kernel<DT, GRAD, NR, SR, TAIL, PASS><<<(uint32_t)grid, 256, 0, st>>>(a, across);
    };
    if constexpr (NR == 8 && !GRAD && (DT == MQ_F32 || SR)) { // (others of that size take the packed kernel)
        // Large inputs of whole lines are read past the caches, which are then left to the codes and to what follows:
        // fp32, with both results read back, 4096 x 4096 46.8 -> 43.5 us, 16384 x 4096 150 -> 135, though alone 71
        // -> 73. Smaller ones may be in the caches already (2048 x 4096 23.8 and 25.2); lines that two rows share
        // are read twice past them (3000 x 3001 30.7 and 36.0). Gradients, of three inputs, lose (102 and 110).
        const int64_t size = DT == MQ_F32 ? 4 : 2;
        const bool whole = (reinterpret_cast<uintptr_t>(a.x.p) | (uint64_t)(a.x.stride * size)) % 64 == 0 && a.cols % 8 == 0;
        if (whole && (int64_t)a.rows * a.cols * size >= 64 << 20) {
            run(Int<0>{}, Int<1>{});
            return hipGetLastError();
        }
    }
    if (a.cols % 8) run(Int<1>{}, Int<0>{});
    else run(Int<0>{}, Int<0>{});
    return hipGetLastError();
}

template <int DT, bool SR>
hipError_t quantize(const Mx4QuantArgs &a, bool grad, hipStream_t st)
{
    if (!grad && !a.col.codes) return rows_alone<DT, SR>(a, st);
    const int height = mx4_quantize_height(a.rows, a.cols, DT, SR, grad);
    if (grad) return height == 8 ? both<DT, true, 8, SR>(a, st) : both<DT, true, 4, SR>(a, st);
    if constexpr (DT != MQ_F32 && !SR)
        if (height == 32) return both<DT, false, 32, SR>(a, st);
    return height == 8 ? both<DT, false, 8, SR>(a, st) : both<DT, false, 4, SR>(a, st);
}

hipError_t quantize(const Mx4QuantArgs &a, bool grad, hipStream_t st)
{
    if (a.x.dtype == MQ_BF16) return a.sr ? quantize<MQ_BF16, true>(a, grad, st) : quantize<MQ_BF16, false>(a, grad, st);
    if (a.x.dtype == MQ_F16) return a.sr ? quantize<MQ_F16, true>(a, grad, st) : quantize<MQ_F16, false>(a, grad, st);
    return a.sr ? quantize<MQ_F32, true>(a, grad, st) : quantize<MQ_F32, false>(a, grad, st);
}

} // namespace

// Rows to a lane. Packed 16-bit elements: 32, of which a column's codes are runs of 16 bytes, where each SIMD has
// a wave (8192 x 4096, 2048 waves, 22.3 us, with 8 rows 26.4; 4096 x 4096, 1024 waves, alone 15.3 and 13.5, but with
// both results read back 36.9 and 39.9: its loads pass the caches, and leave them to what follows). Else 8
// where each SIMD has a wave, 4 below (2048 x 4096 bf16, 2048 waves of 8, 8.3 and 9.2 us, stochastic 16.1 and 17.8;
// 1024 x 2048 4.5 and 4.1, stochastic 9.3 and 7.1). Tiles of 16 rows of fp32 gain nothing: 12288 x 4096 59.2 us where
// 8 rows take 56.3, 3584 x 4096 19.8 and 13.7, with both results read back 107 and 104, 40.7 and 41.0.
int mx4_quantize_height(int rows, int cols, int dtype, bool sr, bool gradients)
{
    const auto waves = [&](int nr) { return ((int64_t)rows + 8 * nr - 1) / (8 * nr) * (((int64_t)cols + 63) / 64); };
    if (dtype != MQ_F32 && !sr && !gradients && waves(32) >= 1024) return 32;
    return waves(8) >= 1024 ? 8 : 4;
}

hipError_t launch_mx4_quantize(const Mx4QuantArgs &a, hipStream_t st) { return quantize(a, false, st); }

hipError_t launch_mx4_gradients(const Mx4QuantArgs &a, hipStream_t st) { return quantize(a, true, st); }

hipError_t launch_mx4_dequantize(const Mx4View &q, const MatView &out, hipStream_t st)
{
    if (q.rows == 0 || q.cols == 0) return hipSuccess;
    const int groups = (q.cols + 7) / 8, width = width_of(groups), across = (groups + width - 1) / width;
    const int64_t grid = ((int64_t)q.rows + 256 / width - 1) / (256 / width) * across;
    if (grid > kMaxGroups) return hipErrorInvalidValue;
    // 16-bit values that would fill the caches are written past them: 8192 x 4096 18.3 -> 16.8 us, 16384 x 4096
    // 47.8 -> 30.9. (Below, the call alone would gain too, 4096 x 4096 11.2 -> 9.7, but what reads the values next
    // would lose as much: both together 21.7 -> 23.1.) A thread's 32 bytes of fp32 leave by two stores, each of
    // every other 16 bytes of a line, which only the caches put together: 16384 x 4096 81 -> 119 us past them.
    const bool through = out.dtype != MQ_F32 && (int64_t)q.rows * q.cols * 2 >= 64 << 20;
    if (out.dtype == MQ_BF16) mx4_dequantize_kernel<MQ_BF16><<<(uint32_t)grid, 256, 0, st>>>(q, out, through, width, across);
    else if (out.dtype == MQ_F16) mx4_dequantize_kernel<MQ_F16><<<(uint32_t)grid, 256, 0, st>>>(q, out, through, width, across);
    else mx4_dequantize_kernel<MQ_F32><<<(uint32_t)grid, 256, 0, st>>>(q, out, through, width, across);
    return hipGetLastError();
}

} // namespace mq
