// mq_mx4_rows.hip -- products of a microscaled 4-bit weight with up to 16 rows.
//
// Bound by the weight's bytes, and by latency where these are few. A workgroup takes 16 of the
// weight's rows; its waves take the pieces of 256 columns in turn, four of them on their way at a
// time, straight into the operand's registers (16x16x128: a lane's 16 bytes are one block, four blocks
// of a row lie beside each other), and their sums are added in LDS, in the waves' order. Where the
// input is small the workgroup quantizes it itself, into LDS, while the weights are on their way: one
// launch, 4096 columns on 4096 rows 5.1 us replayed in place of 6.0. Every workgroup does it, so the
// limit is on all of them together (4 rows of 4096 on 4096 7.0 us, in a launch of its own 6.5, which costs the
// host as much; on 11000 14.2 and 10.4).
// 13 x 8192 on 5120 rows: 10 us of 22.6 MB (2.2 TB/s; 64-column tiles 12); gated 4 x 4096 on 8192: 9.5 us of
// 36 MB (3.8 TB/s). Fewer waves with more pieces each where workgroups are many: 16 waves to each of 1024
// workgroups take 12.6 us where 4 take 9.9.
#include "mq_mx4_device.hpp"

namespace mq {
namespace {

// Piece p of a job's sum: which of its two sums it belongs to, and the place in it.
__device__ __forceinline__ int segment(const Mx4MatmulArgs &a, int &p)
{
    const int s = p >= a.pieces[0];
    p -= s ? a.pieces[0] : 0;
    return s;
}

// The two operands of 128 columns each of a weight's 16 rows: lane (row n, block kb of 4).
struct Strip {
    u32x4_t c[2];
    uint32_t s[2];
};
__device__ __forceinline__ Strip load_strip(const Mx4View &q, int piece, int row, int kb)
{
    const int64_t at = (int64_t)piece * q.rows + row;
    Strip r;
    r.c[0] = *(const u32x4_t *)(q.codes + at * 128 + kb * 16);
    r.c[1] = *(const u32x4_t *)(q.codes + at * 128 + 64 + kb * 16);
    const uint64_t s = *(const uint64_t *)(q.scales + at * 8);
    r.s[0] = (uint32_t)s >> (8 * kb);
    r.s[1] = (uint32_t)(s >> 32) >> (8 * kb);
    return r;
}
__device__ __forceinline__ f32x4_t product16(const Strip &a, const Strip &b, f32x4_t c)
{
    c = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a.c[0]), operand(b.c[0]), c, 4, 4, 0, (int)a.s[0], 0, (int)b.s[0]);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a.c[1]), operand(b.c[1]), c, 4, 4, 0, (int)a.s[1], 0, (int)b.s[1]);
}

// XDT: type of the dense matrix that the workgroup quantizes itself (0: a.a holds it quantized).
template <int DT, bool GATED, int XDT>
__global__ void __launch_bounds__(1024) mx4_rows_kernel(Mx4MatmulArgs a)
{
    constexpr int CH = GATED ? 2 : 4; // pieces on their way at a time
    constexpr int B = GATED ? 2 : 1;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, n = lane & 15, kb = lane >> 4;
    const int job = blockIdx.y, n0 = blockIdx.x * 16;
    const int row = min(n0 + n, a.n - 1), token = min(n, a.m - 1);
    const int total = GATED ? a.pieces[0] : a.pieces[0] + a.pieces[1];
    Strip w[CH][B], x[XDT == 0 ? CH : 1];
    const auto fetch = [&](int p, int i) {
        if (p >= total) return;
        const int s = GATED ? 0 : segment(a, p);
#pragma unroll
        for (int b = 0; b < B; ++b) w[i][b] = load_strip(a.b[job][GATED ? b : s], p, row, kb);
        if constexpr (XDT == 0) x[i] = load_strip(a.a[job][s], p, token, kb);
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) fetch(wave + i * waves, i);

    // x, quantized: codes [piece][row][128], then scales [piece][row][8]
    uint8_t *xs = lds + (size_t)total * a.m * 128;
    if constexpr (XDT != 0) {
        typedef typename Dense<XDT>::T T;
        const T *from = static_cast<const T *>(a.x.p);
        const int groups = total * 32, all = groups * a.m, step = blockDim.x; // of 8 elements; 4 lanes make a block
        for (int i = threadIdx.x; i < all; i += 4 * step) {
            Eight<T> raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = min(i + u * step, all - 1);
                raw[u] = load8<true>(from + j / groups * a.x.stride, reach_of(j % groups * 8, a.cols), a.cols);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u * step >= all) continue;
                const int r = (i + u * step) / groups, g = (i + u * step) % groups, at = (g >> 5) * a.m + r;
                float v[8];
                values8<XDT, true>(raw[u], reach_of(g * 8, a.cols), v);
                const uint32_t e = mx4_scale(quad_max(amax8(v)));
                *(uint32_t *)(lds + at * 128 + (g & 31) * 4) = encode8<false>(v, e, 0, 0, 0, 0);
                if ((g & 3) == 0) xs[at * 8 + (g & 31) / 4] = (uint8_t)e;
            }
        }
        __syncthreads();
    }
    f32x4_t acc[B];
#pragma unroll
    for (int b = 0; b < B; ++b) acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = wave; p < total; p += CH * waves) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int q = p + i * waves;
            if (q < total) {
                if constexpr (XDT != 0) x[0] = load_strip({lds, xs, a.m, 0}, q, token, kb);
#pragma unroll
                for (int b = 0; b < B; ++b) acc[b] = product16(w[i][b], x[XDT == 0 ? i : 0], acc[b]);
            }
            fetch(q + CH * waves, i);
        }
    }
    // lane (n, kb): columns 4 kb .. 4 kb + 3 of row n; the waves' sums in their order
    __syncthreads();
    float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int b = 0; b < B; ++b) *(f32x4_t *)(sums + ((b * waves + wave) * 64 + lane) * 4) = acc[b];
    __syncthreads();
    const int t = threadIdx.x;
    for (int i = t; i < 256; i += blockDim.x) {
        float v[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            v[b] = 0.0f;
            for (int j = 0; j < waves; ++j) v[b] += sums[(b * waves + j) * 256 + i];
        }
        // neighbouring threads: neighbouring columns
        const int l = i / 4, r = l & 15, c = n0 + 4 * (l >> 4) + (i & 3);
        if (r >= a.m || c >= a.n) continue;
        if constexpr (GATED) {
            put<DT>(a.y[0], r, c, silu(v[0]) * v[1]);
            if (a.g.p) {
                put<DT>(a.g, r, c, v[0]);
                put<DT>(a.u, r, c, v[1]);
            }
        } else {
            put<DT>(a.y[job], r, c, v[0]);
        }
    }
}

template <int DT, bool GATED, int XDT>
hipError_t rows(const Mx4MatmulArgs &a, hipStream_t st)
{
    const int total = a.pieces[0] + (GATED ? 0 : a.pieces[1]);
    const dim3 g((a.n + 15) / 16, a.jobs);
    // a wave for each piece, up to 16 of them, while all of the launch's fit the chip
    int waves = 1;
    while (waves < 16 && waves < total && (waves < 4 || (int64_t)waves * 2 * g.x * g.y <= 4096)) waves *= 2;
    const size_t sums = (size_t)waves * 1024 * (GATED ? 2 : 1), x = XDT ? (size_t)total * a.m * 136 : 0;
    mx4_rows_kernel<DT, GATED, XDT><<<g, waves * 64, sums > x ? sums : x, st>>>(a);
    return hipGetLastError();
}

template <int DT, bool GATED>
hipError_t rows(const Mx4MatmulArgs &a, hipStream_t st)
{
    if (a.x.p == nullptr) return rows<DT, GATED, 0>(a, st);
    return a.x.dtype == MQ_BF16 ? rows<DT, GATED, MQ_BF16>(a, st)
                                : (a.x.dtype == MQ_F16 ? rows<DT, GATED, MQ_F16>(a, st) : rows<DT, GATED, MQ_F32>(a, st));
}

template <int DT>
hipError_t rows(const Mx4MatmulArgs &a, hipStream_t st)
{
    return a.gated ? rows<DT, true>(a, st) : rows<DT, false>(a, st);
}

} // namespace

hipError_t launch_mx4_rows(const Mx4MatmulArgs &a, hipStream_t st)
{
    const int dt = a.y[0].dtype;
    return dt == MQ_BF16 ? rows<MQ_BF16>(a, st) : (dt == MQ_F16 ? rows<MQ_F16>(a, st) : rows<MQ_F32>(a, st));
}

} // namespace mq
