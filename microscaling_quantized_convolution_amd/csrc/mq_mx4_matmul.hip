// mq_mx4_matmul.hip -- products of microscaled 4-bit matrices, y = a b^T.
#include "mq_mx4_device.hpp"

namespace mq {
namespace {

// The 16 bytes of one block as an operand: lane (row n, half h) of the 32x32x64 product takes the
// 32 elements of one block, whose scale is byte S of `scales`.
__device__ __forceinline__ i32x8_t operand(u32x4_t c)
{
    return i32x8_t{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

template <int S>
__device__ __forceinline__ f32x16_t product(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb, f32x16_t c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, S, (int)sa, S, (int)sb);
}

// One row's share of a piece for one lane: blocks 4h .. 4h+3 and their scales.
struct Share {
    u32x4_t c[4];
    uint32_t s;
};
__device__ __forceinline__ Share load_share(const Mx4View &q, int piece, int row, int h)
{
    const int64_t at = (int64_t)piece * q.rows + row;
    Share r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.c[i] = *(const u32x4_t *)(q.codes + at * 128 + (4 * h + i) * 16);
    r.s = *(const uint32_t *)(q.scales + at * 8 + 4 * h);
    return r;
}
__device__ __forceinline__ f32x16_t product(const Share &a, const Share &b, f32x16_t c)
{
    c = product<0>(a.c[0], a.s, b.c[0], b.s, c);
    c = product<1>(a.c[1], a.s, b.c[1], b.s, c);
    c = product<2>(a.c[2], a.s, b.c[2], b.s, c);
    return product<3>(a.c[3], a.s, b.c[3], b.s, c);
}

template <int DT>
__device__ __forceinline__ void put(const MatView &y, int64_t r, int c, float v)
{
    static_cast<typename Dense<DT>::T *>(y.p)[r * y.stride + c] = Dense<DT>::store(v);
}

// A wave for each 32 x 32 of the output, operands straight from memory.
template <int DT, bool GATED>
__global__ void __launch_bounds__(256) mx4_matmul_kernel(Mx4MatmulArgs a, int tiles_n)
{
    const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5;
    const int64_t tile = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6);
    const int tm = (int)(tile / tiles_n) * 32, tn = (int)(tile % tiles_n) * 32;
    if (tm >= a.m) return;
    const int job = blockIdx.y;
    const int rm = min(tm + n, a.m - 1), rn = min(tn + n, a.n - 1);
    f32x16_t acc[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.0f;
    for (int p = 0; p < a.pieces[0]; ++p) {
        const Share x = load_share(a.a[job][0], p, rm, h);
        acc[0] = product(x, load_share(a.b[job][0], p, rn, h), acc[0]);
        if constexpr (GATED) acc[1] = product(x, load_share(a.b[job][1], p, rn, h), acc[1]);
    }
    if constexpr (!GATED)
        for (int p = 0; p < a.pieces[1]; ++p)
            acc[0] = product(load_share(a.a[job][1], p, rm, h), load_share(a.b[job][1], p, rn, h), acc[0]);
    if (tn + n >= a.n) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int r = tm + 8 * (i / 4) + 4 * h + i % 4;
        if (r >= a.m) continue;
        if constexpr (GATED) {
            const float g = acc[0][i], u = acc[1][i];
            put<DT>(a.y[0], r, tn + n, g * sigmoid(g) * u);
            if (a.g.p) put<DT>(a.g, r, tn + n, g);
            if (a.u.p) put<DT>(a.u, r, tn + n, u);
        } else {
            put<DT>(a.y[job], r, tn + n, acc[0][i]);
        }
    }
}

template <int DT>
hipError_t matmul(const Mx4MatmulArgs &a, hipStream_t st)
{
    const int tiles_n = (a.n + 31) / 32;
    const int64_t grid = ((int64_t)((a.m + 31) / 32) * tiles_n + 3) / 4;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    const dim3 g((uint32_t)grid, a.jobs);
    if (a.gated) mx4_matmul_kernel<DT, true><<<g, 256, 0, st>>>(a, tiles_n);
    else mx4_matmul_kernel<DT, false><<<g, 256, 0, st>>>(a, tiles_n);
    return hipGetLastError();
}

} // namespace

size_t mx4_matmul_workspace(int, int, int, int) { return 0; }

hipError_t launch_mx4_matmul(const Mx4MatmulArgs &a, hipStream_t st)
{
    if (a.m == 0 || a.n == 0) return hipSuccess;
    return a.y[0].dtype == MQ_BF16 ? matmul<MQ_BF16>(a, st)
                                   : (a.y[0].dtype == MQ_F16 ? matmul<MQ_F16>(a, st) : matmul<MQ_F32>(a, st));
}

} // namespace mq
