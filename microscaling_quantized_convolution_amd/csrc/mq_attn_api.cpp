// mq_attn_api.cpp -- C ABI of the attention and key/value cache calls: host-side validation.
//
// As in mq_api.cpp, every call validates its arguments on the host, then enqueues kernels on the
// caller's stream; nothing here allocates, synchronizes or reads device memory.
#include "mq_attn.hpp"

namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr int32_t kMaxTokens = 1 << 30; // positions of a sequence stay below this
constexpr int64_t kMaxStride = 1 << 24; // 64 rows of keys or values span less than 2^31 bytes

// The kernels number a cache's blocks in 32 bits.
bool blocks_ok(const mq_kv_cache *c)
{
    return (int64_t)c->num_pages * c->kv_heads <= INT32_MAX / (c->page_size / MQ_KV_BLOCK);
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool dim_ok(int32_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

bool cache_ok(const mq_kv_cache *c)
{
    return c && c->num_pages > 0 && c->page_size > 0 && c->page_size % MQ_KV_BLOCK == 0 &&
           c->kv_heads > 0 && c->head_dim > 0 && c->k_codes && c->v_codes && c->k_scales &&
           c->v_scales && aligned(c->k_codes, 16) && aligned(c->v_codes, 16);
}

// Rows are read and written 16 bytes at a time; a tensor without rows may be null.
bool rows_ok(const mq_rows *r)
{
    return r && r->tokens >= 0 && r->heads > 0 && r->head_dim > 0 &&
           (r->dtype == MQ_F16 || r->dtype == MQ_BF16) && (r->data || r->tokens == 0) &&
           aligned(r->data, 16) && r->token_stride >= 0 && r->head_stride >= 0 &&
           r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}

bool ints_ok(const int32_t *p, int64_t n) { return n == 0 || (p && aligned(p, 4)); }

mq::KvView view(const mq_kv_cache *c)
{
    uint32_t shift = 0;
    while (((int64_t)1 << shift) < c->page_size) ++shift;
    const uint64_t mul = ((uint64_t)1 << (31 + shift)) / (uint32_t)c->page_size + 1;
    return {c->k_codes, c->v_codes, c->k_scales, c->v_scales, c->num_pages, c->page_size,
            c->kv_heads, (uint32_t)mul, shift};
}

mq::RowsView view(const mq_rows *r)
{
    return {static_cast<const uint16_t *>(r->data), r->token_stride, r->head_stride};
}

mq_status launched(hipError_t e)
{
    return e == hipSuccess ? MQ_OK : (e == hipErrorInvalidValue ? MQ_ERR_UNSUPPORTED : MQ_ERR_LAUNCH);
}

bool same(const mq_rows *a, const mq_rows *b)
{
    return a->tokens == b->tokens && a->head_dim == b->head_dim && a->dtype == b->dtype;
}

} // namespace

extern "C" {

mq_status mq_kv_append(const mq_kv_cache *cache, const mq_rows *k, const mq_rows *v,
                       const int32_t *table, const int32_t *lens, const int32_t *cu,
                       int32_t n_seqs, int32_t max_pages, hipStream_t stream)
{
    if (!cache_ok(cache) || !rows_ok(k) || !rows_ok(v) || n_seqs < 0 || max_pages < 0) return MQ_ERR_ARG;
    if (!ints_ok(table, (int64_t)n_seqs * max_pages) || !ints_ok(lens, n_seqs) || !ints_ok(cu, n_seqs))
        return MQ_ERR_ARG;
    if (!same(k, v) || k->heads != v->heads || k->heads != cache->kv_heads || k->head_dim != cache->head_dim)
        return MQ_ERR_SHAPE;
    if (!dim_ok(cache->head_dim) || !blocks_ok(cache) || (int64_t)max_pages * cache->page_size > kMaxTokens) return MQ_ERR_UNSUPPORTED;
    if (n_seqs == 0 || max_pages == 0 || k->tokens == 0) return MQ_OK;
    const mq::AppendArgs a = {view(cache), view(k), view(v), table, lens, cu, n_seqs, max_pages, k->tokens};
    return launched(mq::launch_kv_append(a, cache->head_dim, k->dtype, stream));
}

size_t mq_attn_cached_workspace_bytes(int32_t n_seqs, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, int32_t q_len, int32_t max_len,
                                      int32_t weights)
{
    if (n_seqs < 1 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || !dim_ok(head_dim) ||
        q_len < 1 || max_len < 0 || max_len > kMaxTokens || (weights != 0 && weights != 1) ||
        (int64_t)(q_heads / kv_heads) * q_len > INT32_MAX - 16)
        return 0;
    return mq::attn_cached_workspace(n_seqs, q_heads, kv_heads, head_dim, q_len, max_len, weights != 0);
}

mq_status mq_attn_cached(const mq_kv_cache *cache, const mq_rows *q, const mq_rows *out,
                         const int32_t *table, const int32_t *lens, int32_t n_seqs,
                         int32_t max_pages, int32_t q_len, int32_t max_len, float scale,
                         float *weights, void *ws, size_t ws_bytes, hipStream_t stream)
{
    if (!cache_ok(cache) || !rows_ok(q) || !rows_ok(out) || n_seqs < 0 || max_pages < 0 || q_len < 1 ||
        max_len < 0 || !aligned(weights, 4) || !aligned(ws, 16))
        return MQ_ERR_ARG;
    if (!ints_ok(table, (int64_t)n_seqs * max_pages) || !ints_ok(lens, n_seqs)) return MQ_ERR_ARG;
    if (!same(q, out) || q->heads != out->heads || q->head_dim != cache->head_dim ||
        q->heads % cache->kv_heads || (int64_t)n_seqs * q_len != q->tokens)
        return MQ_ERR_SHAPE;
    const int64_t cap = (int64_t)max_pages * cache->page_size;
    const int64_t top = max_len ? max_len : cap;
    if (!dim_ok(cache->head_dim) || !blocks_ok(cache) || cap > kMaxTokens || top > kMaxTokens ||
        (int64_t)(q->heads / cache->kv_heads) * q_len > INT32_MAX - 16)
        return MQ_ERR_UNSUPPORTED;
    if (n_seqs == 0) return MQ_OK;
    const size_t need = mq::attn_cached_workspace(n_seqs, q->heads, cache->kv_heads, cache->head_dim, q_len,
                                                  (int32_t)top, weights != nullptr);
    if (need && (!ws || ws_bytes < need)) return MQ_ERR_WORKSPACE;
    const mq::CachedArgs a = {view(cache), view(q), static_cast<uint16_t *>(out->data), out->token_stride,
                              out->head_stride, table, lens, weights, ws, n_seqs, max_pages, q_len,
                              (int32_t)top, q->heads, (float)(scale * kLog2e)};
    return launched(mq::launch_attn_cached(a, cache->head_dim, q->dtype, stream));
}

mq_status mq_attn_prompt(const mq_rows *q, const mq_rows *k, const mq_rows *v, const mq_rows *out,
                         const int32_t *cu, int32_t n_seqs, int32_t max_len, float scale,
                         hipStream_t stream)
{
    if (!rows_ok(q) || !rows_ok(k) || !rows_ok(v) || !rows_ok(out) || n_seqs < 0 || max_len < 0 ||
        !ints_ok(cu, n_seqs))
        return MQ_ERR_ARG;
    if (!same(q, k) || !same(q, v) || !same(q, out) || q->heads != out->heads || k->heads != v->heads ||
        q->heads % k->heads)
        return MQ_ERR_SHAPE;
    if (!dim_ok(q->head_dim) || max_len > kMaxTokens || k->token_stride > kMaxStride || v->token_stride > kMaxStride)
        return MQ_ERR_UNSUPPORTED;
    const mq::PromptArgs a = {view(q), view(k), view(v), static_cast<uint16_t *>(out->data), out->token_stride,
                              out->head_stride, cu, n_seqs, max_len, q->heads, k->heads, q->tokens,
                              (float)(scale * kLog2e), 0, 0};
    return launched(mq::launch_attn_prompt(a, q->head_dim, q->dtype, stream));
}

mq_status mq_kv_evict(const mq_kv_cache *cache, float *weights, const int32_t *table,
                      const int32_t *lens, const int32_t *new_table, int32_t *new_lens,
                      int32_t *kept, int32_t n_seqs, int32_t max_pages, int32_t new_max_pages,
                      int32_t keep, int32_t recent, hipStream_t stream)
{
    if (!cache_ok(cache) || !weights || !aligned(weights, 4) || n_seqs < 0 || max_pages < 0 ||
        new_max_pages < 0 || keep < 0 || recent < 0)
        return MQ_ERR_ARG;
    if (!ints_ok(table, (int64_t)n_seqs * max_pages) || !ints_ok(lens, n_seqs) ||
        !ints_ok(new_table, (int64_t)n_seqs * new_max_pages) || !ints_ok(new_lens, n_seqs) ||
        !ints_ok(kept, (int64_t)n_seqs * keep) || (n_seqs && new_lens == lens))
        return MQ_ERR_ARG;
    if (keep > (int64_t)new_max_pages * cache->page_size) return MQ_ERR_SHAPE;
    if (!dim_ok(cache->head_dim) || !blocks_ok(cache) || (int64_t)max_pages * cache->page_size > kMaxTokens ||
        keep > kMaxTokens)
        return MQ_ERR_UNSUPPORTED;
    if (n_seqs == 0) return MQ_OK;
    const mq::EvictArgs a = {view(cache), weights, table, lens, new_table, new_lens, kept, n_seqs,
                             max_pages, new_max_pages, keep, recent};
    return launched(mq::launch_kv_evict(a, cache->head_dim, stream));
}

} // extern "C"
