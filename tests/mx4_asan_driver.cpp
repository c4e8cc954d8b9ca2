// mx4_asan_driver.cpp -- the 4-bit layers' host-side validation under AddressSanitizer and
// UndefinedBehaviorSanitizer (test infrastructure, CPU only). Built with g++ together with
// csrc/mq_mx4_api.cpp; the launchers are stubs that check what they are given.
#include "../microscaling_quantized_convolution_amd/csrc/mq_mx4.hpp"

#include <climits>
#include <cstdio>

static int g_launches = 0, g_fail = 0;
static const uint8_t *g_from, *g_to; // the workspace of the call

static void inside(const mq::Mx4View &q)
{
    const size_t rows = (size_t)q.rows * q.pieces();
    if (q.codes >= g_from && q.codes <= g_to && rows &&
        (q.codes + rows * 128 > g_to || q.scales < q.codes + rows * 128 || q.scales + rows * 8 > g_to ||
         (reinterpret_cast<uintptr_t>(q.codes) & 15) || (reinterpret_cast<uintptr_t>(q.scales) & 7)))
        ++g_fail;
}

namespace mq {
hipError_t launch_mx4_quantize(const Mx4QuantArgs &a, hipStream_t) { inside(a.row), inside(a.col); ++g_launches; return hipSuccess; }
hipError_t launch_mx4_gradients(const Mx4QuantArgs &a, hipStream_t)
{
    inside(a.row), inside(a.col), inside(a.row2), inside(a.col2);
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_mx4_dequantize(const Mx4View &, const MatView &, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
hipError_t launch_mx4_matmul(const Mx4MatmulArgs &a, hipStream_t)
{
    for (int j = 0; j < a.jobs; ++j) inside(a.a[j][0]), inside(a.a[j][1]);
    ++g_launches;
    return hipSuccess;
}
bool mx4_quantizes_rows(int m, int, int) { return m == 1; }
size_t mx4_matmul_workspace(int, int, int, int) { return 64; }
} // namespace mq

#define EXPECT(call, st)                                                                       \
    do {                                                                                       \
        const mq_status got_ = (call);                                                         \
        if (got_ != (st)) {                                                                    \
            std::fprintf(stderr, "line %d: %s -> %d\n", __LINE__, #call, (int)got_);           \
            ++g_fail;                                                                          \
        }                                                                                      \
    } while (0)

int main()
{
    uint8_t *p = reinterpret_cast<uint8_t *>(0x10000), *ws = reinterpret_cast<uint8_t *>(0x10000000000);
    hipStream_t st = nullptr;
    const int sizes[] = {0, 1, 3, 255, 256, 257, 1000, 70000, (1 << 30) - 1};
    for (int m : sizes)
        for (int n : sizes)
            for (int k : sizes) {
                const mq_matrix x = {p, k, m, k, MQ_BF16}, y = {p, n, m, n, MQ_F32}, w = {p, k, n, k, MQ_F16};
                const mq_mx4 qw = {n, k, p, p}, qwc = {k, n, p, p}, qxc = {k, m, p, p};
                const auto space = [&](size_t bytes) { g_from = ws, g_to = ws + bytes; return bytes; };
                size_t b = space(mq_mx4_linear_workspace_bytes(m, n, k));
                EXPECT(mq_mx4_linear(&x, &qw, &y, &qxc, ws, b, st), MQ_OK);
                EXPECT(mq_mx4_linear(&x, &qw, &y, nullptr, ws, b, st), MQ_OK);
                b = space(mq_mx4_linear_backward_workspace_bytes(m, n, k));
                EXPECT(mq_mx4_linear_backward(&y, &qxc, &qwc, &x, &w, MQ_SR, 1, ws, b, st), MQ_OK);
                b = space(mq_mx4_gated_workspace_bytes(m, n, k));
                EXPECT(mq_mx4_gated(&x, &qw, &qw, &y, &y, &y, &qxc, ws, b, st), MQ_OK);
                b = space(mq_mx4_gated_backward_workspace_bytes(m, n, k));
                EXPECT(mq_mx4_gated_backward(&y, &y, &y, &qxc, &qwc, &qwc, &x, &w, &w, MQ_RNE, 1, ws, b, st), MQ_OK);
            }
    // extreme sizes in every field, none of which may overflow on the way to a status
    const int odd[] = {INT_MAX, INT_MAX - 255, 1 << 30, 65536, 1, 0, -1, INT_MIN};
    for (int a : odd)
        for (int b : odd)
            for (int c : odd) {
                const mq_matrix x = {p, a, b, c, MQ_F32}, y = {p, INT64_MAX, c, a, MQ_BF16};
                const mq_mx4 q = {a, b, p, p}, r = {c, b, p, p};
                g_from = ws, g_to = ws + ((size_t)1 << 62);
                (void)mq_mx4_quantize(&x, &q, &r, MQ_SR, ~0ull, st);
                (void)mq_mx4_dequantize(&q, &y, st);
                (void)mq_mx4_matmul(&q, &r, &x, ws, (size_t)1 << 62, st);
                (void)mq_mx4_linear(&x, &q, &y, &r, ws, (size_t)1 << 62, st);
                (void)mq_mx4_linear_backward(&x, &q, &r, &y, &x, MQ_SR, 0, ws, (size_t)1 << 62, st);
                (void)mq_mx4_gated(&x, &q, &r, &y, &x, &y, &q, ws, (size_t)1 << 62, st);
                (void)mq_mx4_gated_backward(&x, &y, &x, &q, &r, &q, &x, &y, &y, MQ_RNE, 0, ws, (size_t)1 << 62, st);
                (void)mq_mx4_codes_bytes(a, b);
                (void)mq_mx4_scales_bytes(a, b);
                (void)mq_mx4_gated_backward_workspace_bytes(a, b, c);
            }
    // a launch that does not fit is reported as unsupported
    const mq_matrix x = {p, 8, 4, 8, MQ_F16};
    const mq_mx4 q = {4, 8, p, p};
    EXPECT(mq_mx4_dequantize(&q, &x, st), MQ_ERR_UNSUPPORTED);
    std::printf("%d launches, %d failures\n", g_launches, g_fail);
    return g_fail != 0;
}
