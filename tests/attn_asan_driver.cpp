// attn_asan_driver.cpp -- the attention calls' host-side validation under AddressSanitizer and
// UndefinedBehaviorSanitizer (test infrastructure, CPU only). Built with g++ together with
// csrc/mq_attn_api.cpp; the launchers are stubs that check what they are given.
#include "../microscaling_quantized_convolution_amd/csrc/mq_attn.hpp"

#include <climits>
#include <cstdio>

static int g_launches = 0, g_fail = 0;

static void check_page(const mq::KvView &c)
{
    // the multiplication that stands for a division by the page size, at its edges
    const uint32_t at[] = {0u, 1u, (uint32_t)c.page - 1, (uint32_t)c.page, (uint32_t)c.page + 1, 1u << 30,
                           (1u << 30) / c.page * c.page, (1u << 30) / c.page * c.page - 1, 0x7fffffffu};
    for (uint32_t t : at)
        if (((uint64_t)t * c.page_mul >> (31 + c.page_shift)) != t / (uint32_t)c.page) {
            std::fprintf(stderr, "page %d: %u / %d\n", c.page, t, c.page);
            ++g_fail;
        }
}

namespace mq {
hipError_t launch_kv_append(const AppendArgs &a, int, int, hipStream_t) { check_page(a.c); ++g_launches; return hipSuccess; }
hipError_t launch_kv_evict(const EvictArgs &a, int, hipStream_t) { check_page(a.c); ++g_launches; return hipSuccess; }
size_t attn_cached_workspace(int, int, int, int, int, int, bool) { return 4096; }
hipError_t launch_attn_cached(const CachedArgs &a, int, int, hipStream_t) { check_page(a.c); ++g_launches; return hipSuccess; }
hipError_t launch_attn_prompt(const PromptArgs &, int, int, hipStream_t) { ++g_launches; return hipErrorInvalidValue; }
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
    uint8_t *p = reinterpret_cast<uint8_t *>(0x10000);
    int32_t *i = reinterpret_cast<int32_t *>(0x20000), *i2 = i + 1024;
    float *f = reinterpret_cast<float *>(0x30000);
    hipStream_t st = nullptr;
    for (int page = 16; page <= 4096; page += 16) {
        const mq_kv_cache c = {4, page, 2, 64, p, p, p, p};
        const mq_rows r = {p, 128, 64, 4, 2, 64, MQ_F16}, q = {p, 256, 64, 4, 4, 64, MQ_F16};
        EXPECT(mq_kv_append(&c, &r, &r, i, i, i, 2, 3, st), MQ_OK);
        EXPECT(mq_attn_cached(&c, &q, &q, i, i, 2, 3, 2, 0, 1.0f, f, p, 4096, st), MQ_OK);
        EXPECT(mq_kv_evict(&c, f, i, i, i, i2, i, 2, 3, 3, 16, 4, st), MQ_OK);
    }
    // extreme sizes in every field, none of which may overflow on the way to a status
    const int odd[] = {INT_MAX, INT_MAX - 15, 1 << 30, 65536, 16, 1, 0, -1, INT_MIN};
    for (int a : odd)
        for (int b : odd) {
            const mq_kv_cache c = {a, b, b, 64, p, p, p, p};
            const mq_kv_cache d = {4, 32, a, b, p, p, p, p};
            const mq_rows r = {p, a, b, a, b, 64, MQ_BF16}, q = {p, 8, 8, b, a, 128, MQ_F16};
            const mq_rows s = {p, INT64_MAX - 7, INT64_MIN, a, 2, 64, MQ_F16};
            (void)mq_kv_append(&c, &r, &r, i, i, i, a, b, st);
            (void)mq_kv_append(&d, &q, &q, i, i, i, b, a, st);
            (void)mq_attn_cached(&c, &r, &r, i, i, b, a, a, b, 1.0f, f, p, 4096, st);
            (void)mq_attn_cached(&d, &q, &q, i, i, a, b, b, a, 1.0f, nullptr, nullptr, 0, st);
            (void)mq_attn_prompt(&r, &q, &q, &r, i, a, b, 1.0f, st);
            (void)mq_attn_prompt(&s, &s, &s, &s, i, b, a, 1.0f, st);
            (void)mq_kv_evict(&c, f, i, i, i, i2, i, a, b, a, b, a, st);
            (void)mq_kv_evict(&d, f, i, i, i, i2, i, b, a, b, a, b, st);
            (void)mq_attn_cached_workspace_bytes(a, b, a, 64, b, a, 1);
            (void)mq_attn_cached_workspace_bytes(1, a, 1, 128, b, a, 0);
        }
    // a launch that does not fit is reported as unsupported
    const mq_rows r = {p, 128, 64, 4, 2, 64, MQ_F16};
    EXPECT(mq_attn_prompt(&r, &r, &r, &r, i, 1, 4, 1.0f, st), MQ_ERR_UNSUPPORTED);
    std::printf("%d launches, %d failures\n", g_launches, g_fail);
    return g_fail != 0;
}
