// mq_mx4_quantize.hip -- microscaled 4-bit quantization along rows and columns, and back.
#include "mq_mx4_device.hpp"

namespace mq {
namespace {

// One of the values that are quantized: an element of x, or of a gradient of h = silu(g) u.
enum { kPlain, kGradG, kGradU };
template <int DT, int KIND>
__device__ __forceinline__ float value_at(const Mx4QuantArgs &a, int r, int c)
{
    typedef typename Dense<DT>::T T;
    const auto at = [&](const MatView &m) { return Dense<DT>::load(static_cast<const T *>(m.p)[r * m.stride + c]); };
    const float x = at(a.x);
    if constexpr (KIND == kPlain) return x;
    const float g = at(a.g), s = sigmoid(g);
    if constexpr (KIND == kGradU) return x * (g * s);
    return x * at(a.u) * (s * (1.0f + g * (1.0f - s)));
}

// A thread for each block of 32, the blocks that fill up the last piece included.
template <int DT, int KIND, bool COL, bool SR>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(Mx4QuantArgs a, Mx4View q)
{
    const int pieces = q.pieces();
    const int64_t id = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (id >= (int64_t)q.rows * pieces * 8) return;
    // neighbouring threads read neighbouring elements
    const int r = COL ? (int)(id % q.rows) : (int)(id / (pieces * 8));
    const int b = COL ? (int)(id / q.rows) : (int)(id % (pieces * 8));
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int c = b * 32 + j;
        v[j] = c < q.cols ? (COL ? value_at<DT, KIND>(a, c, r) : value_at<DT, KIND>(a, r, c)) : 0.0f;
    }
    const uint64_t t = (uint64_t)r * (uint32_t)((q.cols + 31) / 32) + b;
    u32x4_t codes;
    const uint32_t e = mx4_block<SR>(v, t, (COL ? 1u : 0u) + (KIND == kGradU ? 2u : 0u), a.seed_lo, a.seed_hi, &codes);
    const int64_t at = ((int64_t)(b / 8) * q.rows + r) * 8 + b % 8;
    *(u32x4_t *)(q.codes + at * 16) = codes;
    q.scales[at] = (uint8_t)e;
}

template <int DT>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(Mx4View q, MatView out)
{
    const int blocks = (q.cols + 31) / 32;
    const int64_t id = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (id >= (int64_t)q.rows * blocks) return;
    const int r = (int)(id / blocks), b = (int)(id % blocks);
    const int64_t at = ((int64_t)(b / 8) * q.rows + r) * 8 + b % 8;
    const u32x4_t codes = *(const u32x4_t *)(q.codes + at * 16);
    const uint32_t e = q.scales[at];
    typedef typename Dense<DT>::T T;
    T *to = static_cast<T *>(out.p) + r * out.stride + b * 32;
    for (int j = 0; j < 32 && b * 32 + j < q.cols; ++j) {
        const uint32_t c = codes[j / 8] >> (4 * (j % 8));
        const float m = elem_mag_to_float<kFP4>(c & 7u);
        const float v = __builtin_amdgcn_ldexpf(c & 8u ? -m : m, (int)e - 127);
        to[j] = Dense<DT>::store(e == 255 ? __uint_as_float(0x7FC00000u) : v);
    }
}

template <int DT, int KIND, bool COL>
hipError_t quantize(const Mx4QuantArgs &a, const Mx4View &q, hipStream_t st)
{
    if (!q.codes) return hipSuccess;
    const int64_t threads = (int64_t)q.rows * q.pieces() * 8, grid = (threads + 255) / 256;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (a.sr) mx4_quantize_kernel<DT, KIND, COL, true><<<(uint32_t)grid, 256, 0, st>>>(a, q);
    else mx4_quantize_kernel<DT, KIND, COL, false><<<(uint32_t)grid, 256, 0, st>>>(a, q);
    return hipGetLastError();
}

template <int DT>
hipError_t gradients(const Mx4QuantArgs &a, hipStream_t st)
{
    hipError_t e = quantize<DT, kGradG, false>(a, a.row, st);
    if (e == hipSuccess) e = quantize<DT, kGradU, false>(a, a.row2, st);
    if (e == hipSuccess) e = quantize<DT, kGradG, true>(a, a.col, st);
    if (e == hipSuccess) e = quantize<DT, kGradU, true>(a, a.col2, st);
    return e;
}

template <int DT>
hipError_t plain(const Mx4QuantArgs &a, hipStream_t st)
{
    const hipError_t e = quantize<DT, kPlain, false>(a, a.row, st);
    return e == hipSuccess ? quantize<DT, kPlain, true>(a, a.col, st) : e;
}

} // namespace

hipError_t launch_mx4_quantize(const Mx4QuantArgs &a, hipStream_t st)
{
    return a.x.dtype == MQ_BF16 ? plain<MQ_BF16>(a, st) : (a.x.dtype == MQ_F16 ? plain<MQ_F16>(a, st) : plain<MQ_F32>(a, st));
}

hipError_t launch_mx4_gradients(const Mx4QuantArgs &a, hipStream_t st)
{
    return a.x.dtype == MQ_BF16 ? gradients<MQ_BF16>(a, st)
                                : (a.x.dtype == MQ_F16 ? gradients<MQ_F16>(a, st) : gradients<MQ_F32>(a, st));
}

hipError_t launch_mx4_dequantize(const Mx4View &q, const MatView &out, hipStream_t st)
{
    const int64_t threads = (int64_t)q.rows * ((q.cols + 31) / 32), grid = (threads + 255) / 256;
    if (grid == 0) return hipSuccess;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    if (out.dtype == MQ_BF16) mx4_dequantize_kernel<MQ_BF16><<<(uint32_t)grid, 256, 0, st>>>(q, out);
    else if (out.dtype == MQ_F16) mx4_dequantize_kernel<MQ_F16><<<(uint32_t)grid, 256, 0, st>>>(q, out);
    else mx4_dequantize_kernel<MQ_F32><<<(uint32_t)grid, 256, 0, st>>>(q, out);
    return hipGetLastError();
}

} // namespace mq
