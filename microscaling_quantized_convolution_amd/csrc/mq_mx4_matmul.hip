// mq_mx4_matmul.hip -- products of microscaled 4-bit matrices, y = a b^T.
//
// y[m][n] = sum over blocks of 2^(ea + eb) sum over their 32 elements of a[m][k] b[n][k]: the scaled
// matrix instruction (32x32x64, 4-bit operands, two blocks' scales to each row) takes codes and scale
// bytes as they lie in memory and adds up in fp32, exactly but for the additions' rounding.
//
// A workgroup holds a tile of the output in registers and passes over the pieces of 256 columns. A
// piece of its rows is contiguous in memory; it goes straight into a ring of slots in LDS
// (global_load_lds, no registers between), scales with it, and the slot that a piece has left is
// loaded with the piece STAGES - 1 ahead. A lane takes blocks 4h .. 4h+3 of its row one after the other
// (h its half of the wave), so one word of scales serves its four products. The weight's rows are the
// instruction's rows and the tokens its columns: a lane's accumulators are then runs of four
// columns of one output row.
//
// Tiles, and the launches' times (us, replayed from graphs, bf16 out; m x n x k):
//   64 x 64, 4 slots, two workgroups a CU     small outputs: latency counts, and the number of workgroups.
//                                             256 x 4096 x 4096 7.9 (128 x 128 12.6, 256 x 256 26)
//   128 x 128, 4 slots                        up to one tile to a CU: 1024 x 4096 x 4096 15.1 (2 slots 15.9)
//   128 x 128, 2 slots, two workgroups a CU   one's stores under the other's products: 4096 x 4096 x 512 13.1
//   256 x 256, 2 slots                        8192 x 8192 x 4096 144 (3.8 PFLOP/s), x 16384 504 (4.36)
// Bound at 256 x 256, for each piece of 1.81 us: the matrix instructions 0.98 (8.8 PFLOP/s on all CUs), but
// on random data the clock falls, and products with their LDS reads alone take 1.47 (1.12 on zeros); the 68 KB of
// a piece 0.98 where two pieces are on their way, 1.36 where one is and 0.6 from L2. A third slot has no room
// beside 64 KB, smaller tiles load more (256 x 128 with three slots: 45 us at 4096 x 4096 x 4096 against 37).
// Scales by loads of their own to registers cost 0.29; a piece's loads spread over its products arrive too
// late (524 to 559 us). Persistent workgroups that load the next tile before they store this one gained
// nothing: stores to memory were the limit, and writing large outputs past the caches is what moved it.
#include "mq_mx4_device.hpp"

#include <type_traits>
#include <utility>

namespace mq {
namespace {

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

// The same, 64 lanes x 4 bytes to 256 bytes of LDS.
__device__ __forceinline__ void load_word_to_lds(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory");
}

// All but the wave's last LEFT loads into LDS have arrived, every read of LDS is done, for all waves.
template <int LEFT>
__device__ __forceinline__ void lds_barrier()
{
    static_assert(LEFT < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\t"
                 "s_barrier" ::"n"(LEFT)
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

__device__ __forceinline__ u32x4_t read_lds(uint32_t at)
{
    typedef const __attribute__((address_space(3))) u32x4_t *lp;
    return *(lp)(uintptr_t)at;
}

__device__ __forceinline__ uint32_t read_lds_word(uint32_t at)
{
    typedef const __attribute__((address_space(3))) uint32_t *lp;
    return *(lp)(uintptr_t)at;
}

// A wave's 32 rows of NT 32 x 32 tiles beside each other, through its own part of LDS: accumulator k of
// lane (n, h) is row n, column 8 (k / 4) + 4 h + k % 4 of its tile, and memory is written in whole rows
// of the strip, 16 bytes to a lane (at any alignment). 16 bytes between the rows keep them in
// different banks.
template <int DT, int NT> struct Strip {
    typedef typename Dense<DT>::T T;
    static constexpr int E = 16 / (int)sizeof(T), ACROSS = NT * 32 / E, stride = ACROSS * 16 + 16, bytes = 32 * stride;
    static __device__ __forceinline__ void put(const MatView &y, uint32_t region, int lane, int r0, int c0, int rows, int cols, bool through, const f32x16_t *v)
    {
        const uint32_t to = region + (lane & 31) * stride + (lane >> 5) * 4 * sizeof(T);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                T e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = Dense<DT>::store(v[j][4 * g + k]);
                const uint32_t at = to + (j * 32 + 8 * g) * sizeof(T);
                if constexpr (sizeof(T) == 4) *(__attribute__((address_space(3))) u32x4_t *)(uintptr_t)at = *(const u32x4_t *)e;
                else *(__attribute__((address_space(3))) uint64_t *)(uintptr_t)at = *(const uint64_t *)e;
            }
        __builtin_amdgcn_wave_barrier(); // (a wave's accesses to LDS are made in their order)
        const int chunk = lane % ACROSS, c = c0 + chunk * E;
#pragma unroll
        for (int i = 0; i < ACROSS / 2; ++i) { // 64 / ACROSS rows at a time
            const int row = i * (64 / ACROSS) + lane / ACROSS, r = r0 + row;
            const u32x4_t x = read_lds(region + row * stride + chunk * 16);
            if (r >= rows) continue;
            T *out = static_cast<T *>(y.p) + r * y.stride + c;
            if (c + E <= cols) {
                if (through) store_past(out, x);
                else *(Sixteen *)out = x;
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (c + k < cols) out[k] = ((const T *)&x)[k];
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    typedef u32x4_t Sixteen __attribute__((aligned(2)));
};

// f(0), ..., f(N - 1), each with its number as a type
template <int N, class F, int... I>
__device__ __forceinline__ void unroll_(F &&f, std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
template <int N, class F>
__device__ __forceinline__ void unroll(F &&f) { unroll_<N>(f, std::make_integer_sequence<int, N>{}); }

// WM x WN waves, each of TM x TN tiles of 32 x 32; STAGES pieces in LDS. Gated: the tile's columns are
// as many of the gate's and of the other factor, a wave holds both for the same outputs.
template <int DT, bool GATED, int WM, int WN, int TM, int TN, int STAGES>
__global__ void __launch_bounds__(WM * WN * 64, WM * WN == 4 && (WM * TM + WN * TN) * 32 * 136 * STAGES > 80 * 1024 ? 1 : 2) mx4_matmul_kernel(Mx4MatmulArgs a, int tiles_m, int tiles_n)
{
    constexpr int W = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
    constexpr int LA = BM / 8 / W, LB = BN / 8 / W; // 1 KB pieces of a stage to each wave
    constexpr int ON = GATED ? BN / 2 : BN;         // output columns of a tile
    constexpr int HALF = TN > 1 ? TN / 2 : 1;       // gated: a wave's gates, whose other factors follow
    constexpr int LZ = (BM + BN + W * 32 - 1) / (W * 32), ZR = LZ * W * 32; // 32 rows' scales to a load; the
                                                                            // last wave's may be no one's
    constexpr int A = 0, B = STAGES * BM * 128, Z = B + STAGES * BN * 128, LDS = Z + STAGES * ZR * 8;
    __shared__ __align__(256) uint8_t lds[LDS];
    static_assert(BM % (W * 8) == 0 && BN % (W * 8) == 0, "the waves' shares are whole");
    static_assert(LA % 2 == 0 && LB % 2 == 0, "every other load takes its blocks 64 bytes on");
    static_assert(BM / 32 % LZ == 0 && ON / 32 % LZ == 0, "a wave's scales are of one operand");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, h = lane >> 5, wm = wave / WN, wn = wave % WN;
    const int job = blockIdx.y;
    // workgroups go to the 8 XCDs in turn: each XCD receives one stretch of the tiles, eight rows of
    // tiles to a band
    int tile = blockIdx.x;
    {
        const int count = tiles_m * tiles_n, per = count / 8, rest = count % 8, x = tile % 8;
        tile = x * per + min(x, rest) + tile / 8;
    }
    constexpr int BAND = 8;
    const int band = tile / (BAND * tiles_n), in = tile % (BAND * tiles_n);
    const int high = min(BAND, tiles_m - band * BAND);
    const int m0 = (band * BAND + in % high) * BM, n0 = in / high * ON;

    // Where the lane's 16 bytes of each 1 KB come from: block (lane % 8) ^ (row / 2 % 8) of its row,
    // so that 16 rows' blocks of one number lie in different banks; the last row again past it.
    const uint32_t block = ((lane & 7) ^ (lane >> 4)) * 16;
    const int b_part = GATED ? wave / (W / 2) : 0, b_wave = GATED ? wave % (W / 2) : wave;
    uint32_t from_a = (wave * LA * 8 + (lane >> 3)) * 128 + block, lim_a = (min(a.m - m0, BM) - 1) * 128 + block;
    uint32_t from_b = (b_wave * LB * 8 + (lane >> 3)) * 128 + block, lim_b = (min(a.n - n0, ON) - 1) * 128 + block;
    const uint32_t lds_a = lds_address(lds) + A, lds_b = lds_address(lds) + B, lds_z = lds_address(lds) + Z;
    // rows of the lane's operands, whose scales it takes four blocks to a word
    const auto b_row = [&](int j) {
        return GATED ? (j / HALF) * ON + (wn * HALF + j % HALF) * 32 : (wn * TN + j) * 32;
    };
    // the wave's share of the scales: 32 rows to a load, 4 blocks to a lane; the first waves take a's
    const int z_row = wave * LZ * 32, z_part = z_row < BM ? 0 : (GATED && z_row >= BM + ON ? 2 : 1);
    const int z_first = z_part == 0 ? z_row : z_row - BM - (z_part == 2 ? ON : 0);
    uint32_t from_z = z_first * 8 + lane * 4, lim_z = (min(z_part == 0 ? a.m - m0 : a.n - n0, z_part == 0 ? BM : ON) - 1) * 8 + (lane & 1) * 4;

    // the piece that is loaded next
    const int total = GATED ? a.pieces[0] : a.pieces[0] + a.pieces[1];
    const uint8_t *ca, *cb, *cz;
    int64_t rows_a, rows_b;
    const auto open = [&](int s) {
        const Mx4View va = a.a[job][s], vb = a.b[job][GATED ? b_part : s];
        rows_a = va.rows;
        rows_b = vb.rows;
        ca = va.codes + (int64_t)m0 * 128;
        cb = vb.codes + (int64_t)n0 * 128;
        cz = z_part == 0 ? va.scales + (int64_t)m0 * 8 : a.b[job][GATED ? z_part - 1 : s].scales + (int64_t)n0 * 8;
    };
    int next = 0;
    const auto advance = [&] {
        ++next;
        if (next >= total) return; // the last piece again: nothing reads it
        if (!GATED && next == a.pieces[0]) return open(1);
        ca += rows_a * 128;
        cb += rows_b * 128;
        cz += (z_part == 0 ? rows_a : rows_b) * 8;
    };
    // load i of the wave's LOADS of the next piece
    constexpr int LOADS = LZ + LA + LB;
    const auto stage = [&](auto ic) {
        constexpr int i = decltype(ic)::value;
        const int slot = next % STAGES;
        if constexpr (i < LZ)
            load_word_to_lds(cz, min(from_z + i * 256, lim_z), lds_z + slot * ZR * 8 + (wave * LZ + i) * 256);
        else if constexpr (i < LZ + LA)
            load_to_lds(ca, min(from_a + (i - LZ) * 1024, lim_a) ^ ((i - LZ) % 2 * 64), lds_a + slot * BM * 128 + (wave * LA + i - LZ) * 1024);
        else
            load_to_lds(cb, min(from_b + (i - LZ - LA) * 1024, lim_b) ^ ((i - LZ - LA) % 2 * 64), lds_b + slot * BN * 128 + (wave * LB + i - LZ - LA) * 1024);
    };
    f32x16_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if (total > 0) {
        open(!GATED && a.pieces[0] == 0);
        unroll<STAGES>([&](auto) {
            unroll<LOADS>(stage);
            advance();
        });
    }
    const auto multiply = [&](int p, auto more) {
        const int at = p % STAGES;
        const uint32_t at_a = lds_a + at * BM * 128 + (wm * TM * 32 + n) * 128;
        const uint32_t at_b = lds_b + at * BN * 128 + n * 128;
        u32x4_t fa[2][TM], fb[2][TN];
        const auto fetch = [&](auto sc) {
            constexpr int S = decltype(sc)::value;
            const uint32_t slot = (uint32_t)((4 * h + S) ^ (n / 2 & 7)) * 16;
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[S & 1][j] = read_lds(at_b + b_row(j) * 128 + slot);
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[S & 1][i] = read_lds(at_a + i * 4096 + slot);
        };
        fetch(std::integral_constant<int, 0>{});
        uint32_t sa[TM], sb[TN];
        const uint32_t at_z = lds_z + at * ZR * 8 + n * 8 + h * 4;
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = read_lds_word(at_z + (BM + b_row(j)) * 8);
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = read_lds_word(at_z + (wm * TM + i) * 256);
        // (the addresses of a piece's loads are made anew: kept, they would not fit)
        asm volatile("" : "+v"(from_a), "+v"(from_b), "+v"(from_z));
        unroll<4>([&](auto sc) {
            constexpr int S = decltype(sc)::value;
            if constexpr (S < 3) fetch(std::integral_constant<int, S + 1>{});
            unroll<TM>([&](auto tc) {
                constexpr int i = decltype(tc)::value;
                unroll<LOADS>([&](auto lc) {
                    constexpr int l = decltype(lc)::value;
                    // early, all in the first step: a barrier soon waits for them
                    if constexpr (decltype(more)::value && l * TM / LOADS == S * TM + i) stage(lc);
                });
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    acc[i][j] = product<S>(fb[S & 1][j], sb[j], fa[S & 1][i], sa[i], acc[i][j]);
                    asm volatile("" : "+v"(acc[i][j])); // here, in the order of the loads
                }
            });
        });
        if constexpr (decltype(more)::value) advance();
    };
    // before each piece: it is there for all waves, and the piece before it is no longer read
    if (total > 0) {
        lds_barrier<(STAGES - 1) * LOADS>();
        multiply(0, std::false_type{});
    }
    for (int p = 1; p < total; ++p) {
        lds_barrier<(STAGES - 2) * LOADS>();
        multiply(p, std::true_type{});
    }
    lds_barrier<0>(); // no load into LDS is left, and all of it is free
    constexpr int NT = GATED ? HALF : TN;
    static_assert(W * Strip<DT, NT>::bytes <= LDS, "a strip of 32 rows to each wave");
    const uint32_t region = lds_address(lds) + wave * Strip<DT, NT>::bytes;
    const int c = n0 + (GATED ? wn * HALF : wn * TN) * 32;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = m0 + (wm * TM + i) * 32;
        if constexpr (GATED) {
            f32x16_t out[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k) out[j][k] = silu(acc[i][j][k]) * acc[i][j + HALF][k];
            Strip<DT, NT>::put(a.y[0], region, lane, r, c, a.m, a.n, a.through, out);
            if (a.g.p) {
                Strip<DT, NT>::put(a.g, region, lane, r, c, a.m, a.n, a.through, acc[i]);
                Strip<DT, NT>::put(a.u, region, lane, r, c, a.m, a.n, a.through, acc[i] + HALF);
            }
        } else {
            Strip<DT, NT>::put(a.y[job], region, lane, r, c, a.m, a.n, a.through, acc[i]);
        }
    }
}

template <int DT, bool GATED, int WM, int WN, int TM, int TN, int STAGES>
hipError_t matmul_tiles(const Mx4MatmulArgs &a, hipStream_t st)
{
    constexpr int BM = WM * TM * 32, BN = WN * TN * 32 / (GATED ? 2 : 1);
    const int tiles_m = (a.m + BM - 1) / BM, tiles_n = (a.n + BN - 1) / BN;
    const int64_t grid = (int64_t)tiles_m * tiles_n;
    if (grid > UINT32_MAX / (WM * WN * 64)) return hipErrorInvalidValue; // a grid's threads are counted in 32 bits
    const dim3 g((uint32_t)grid, a.jobs);
    mx4_matmul_kernel<DT, GATED, WM, WN, TM, TN, STAGES><<<g, WM * WN * 64, 0, st>>>(a, tiles_m, tiles_n);
    return hipGetLastError();
}

template <int DT, bool GATED>
hipError_t matmul(const Mx4MatmulArgs &a, int kind, hipStream_t st)
{
    if (kind == kMx4Tile256) return matmul_tiles<DT, GATED, 4, 2, 2, 4, 2>(a, st);
    if (kind == kMx4Tile128) return matmul_tiles<DT, GATED, 4, 2, 1, 2, 2>(a, st);
    if (kind == kMx4Tile128Deep) return matmul_tiles<DT, GATED, 4, 2, 1, 2, 4>(a, st);
    if constexpr (GATED) return matmul_tiles<DT, true, 2, 2, 1, 2, 3>(a, st);
    else return matmul_tiles<DT, false, 2, 2, 1, 1, 4>(a, st);
}

template <int DT>
hipError_t matmul(const Mx4MatmulArgs &a, int kind, hipStream_t st)
{
    return a.gated ? matmul<DT, true>(a, kind, st) : matmul<DT, false>(a, kind, st);
}

int64_t tiles_of(int jobs, int m, int n, int bm, int bn)
{
    return (((int64_t)m + bm - 1) / bm) * (((int64_t)n + bn - 1) / bn) * jobs;
}

} // namespace

int mx4_matmul_kind(int jobs, int m, int n, int pieces, bool gated)
{
    const auto tiles = [&](int bm, int bn) { return tiles_of(jobs, m, n, bm, bn); };
    if (mx4_takes_rows(m, (int64_t)n * jobs, gated)) return kMx4Rows;
    // 64 x 64 while the chip holds them all at once: 512 x 4096 x 4096 (512 tiles) 10.7 us, 128 x 128 12.8;
    // 1024 x 4096 x 4096 19.1 and 15.1. Gated (twice the weight's rows to a tile), with the quantization: 300 x
    // 1024 on 2700 (215) 7.7 and 8.6, 256 x 4096 on 8192 (512) 19.2 and 17.4.
    if (tiles(64, 64) <= (gated ? 256 : 512)) return kMx4Tile64;
    // four slots while no CU has two of 128 x 128: 2048 x 2048 x 8192 (256) 24.9 us, with two slots 27.1;
    // 2048 x 4096 x 4096 (512) 27.4 and 23.7
    if (tiles(128, gated ? 64 : 128) <= 256) return kMx4Tile128Deep;
    // 256 x 256 one to a CU, or 128 x 128 two to a CU: rounds of the chip, each of so much for a piece
    // and for a tile's beginning and end (in ns, measured at 2 to 64 pieces): 2048 x 4096 x 4096 28.4 and
    // 23.7 us, 4096 x 4096 x 512 13.4 and 13.1, 5000 x 3000 x 4096 36.1 and 43.2, 4096 x 4096 x 16384 131 and 158
    const double t256 = (double)((tiles(256, gated ? 128 : 256) + 255) / 256) * (1810.0 * pieces + 8000);
    const double t128 = (double)((tiles(128, gated ? 64 : 128) + 511) / 512) * (1250.0 * pieces + 3000);
    return t256 < t128 ? kMx4Tile256 : kMx4Tile128;
}

bool mx4_quantizes_rows(int m, int n, int k)
{
    return mx4_takes_rows(m, n, false) && (int64_t)m * k <= 1 << 14 && (int64_t)m * k * ((n + 15) / 16) <= 1 << 22;
}

hipError_t launch_mx4_matmul(const Mx4MatmulArgs &given, hipStream_t st)
{
    if (given.m == 0 || given.n == 0) return hipSuccess;
    Mx4MatmulArgs a = given;
    const int kind = mx4_matmul_kind(a.jobs, a.m, a.n, a.pieces[0] + a.pieces[1], a.gated);
    if (kind == kMx4Rows) return launch_mx4_rows(a, st);
    // Outputs that would fill the caches, and those of many rounds of tiles, are written past them: other
    // tiles' loads then pass the stores (8192 x 8192 x 4096 to bf16 155 -> 144 us, 8192 x 8192 x 512 57 -> 41,
    // gated 4096 x 8192 x 4096 152 -> 139, with G and U 176 -> 159; but 8192 x 4096 x 4096, two rounds of 67
    // MB, 75 -> 78). Rows that share lines of memory leave them half written: only the caches put these
    // together (5000 x 4200 x 1000 to fp32 32 us, past them 36; gated 3000 x 5001 x 1000 with G and U 46,
    // past them 98), until one output alone is far larger than they are, and its sums are long enough to hide it
    // (8192 x 8191 to bf16, 134 MB: of 512 columns 57 and 66 us, of 1024 69 and 66, of 4096 158 and 152).
    const int size = a.y[0].dtype == MQ_F32 ? 4 : 2, outputs = a.jobs + (a.g.p ? 2 : 0);
    const int64_t bytes = (int64_t)a.m * a.n * size * outputs;
    const auto whole = [&](const MatView &y) { return (reinterpret_cast<uintptr_t>(y.p) | (uint64_t)y.stride * size) % 64 == 0; };
    if (whole(a.y[0]) && whole(a.y[1]) && whole(a.g) && whole(a.u)) // (those that are not wanted are 0)
        a.through = bytes >= 80 << 20 || (kind == kMx4Tile256 && tiles_of(a.jobs, a.m, a.n, 256, a.gated ? 128 : 256) >= 768);
    else
        a.through = outputs == 1 && bytes >= 112 << 20 && a.pieces[0] + a.pieces[1] >= 4;
    const int dt = a.y[0].dtype;
    return dt == MQ_BF16 ? matmul<MQ_BF16>(a, kind, st) : (dt == MQ_F16 ? matmul<MQ_F16>(a, kind, st) : matmul<MQ_F32>(a, kind, st));
}

} // namespace mq
