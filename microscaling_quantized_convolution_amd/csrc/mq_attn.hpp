// mq_attn.hpp -- what the attention and key/value cache kernels share (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mq.h"

namespace mq {

constexpr int kKvBlock = MQ_KV_BLOCK; // tokens per scale
constexpr int kScaleMin = 10;         // smallest scale byte written: the step of the smallest
                                      // codes, 2^-9 * 2^(10-127), is the smallest normal fp32

// A paged cache (mq_kv_cache; head_dim is a template parameter of the kernels). A position t is
// divided by the page size as t * page_mul >> (31 + page_shift): with s = ceil(log2 page) and
// mul = floor(2^(31+s) / page) + 1, mul * page exceeds 2^(31+s) by at most page <= 2^s, so the
// quotient is exact for every t < 2^31.
struct KvView {
    uint8_t *kc, *vc, *ks, *vs;
    int pages, page, heads;
    uint32_t page_mul, page_shift;
};

// Token vectors (mq_rows; strides in elements).
struct RowsView {
    const uint16_t *p;
    int64_t ts, hs;
};

struct AppendArgs {
    KvView c;
    RowsView k, v;
    const int32_t *table, *lens, *cu;
    int n, max_pages, total;
};

struct EvictArgs {
    KvView c;
    float *weights;
    const int32_t *table, *lens, *new_table;
    int32_t *new_lens, *kept;
    int n, max_pages, new_max_pages, keep, recent;
};

struct CachedArgs {
    KvView c;
    RowsView q;
    uint16_t *out;
    int64_t out_ts, out_hs;
    const int32_t *table, *lens;
    float *weights; // null: none
    void *ws;
    int n, max_pages, q_len, max_len, q_heads;
    float scale_log2e; // softmax scale times log2(e)
};

struct PromptArgs {
    RowsView q, k, v;
    uint16_t *out;
    int64_t out_ts, out_hs;
    const int32_t *cu;
    int n, max_len, q_heads, kv_heads, total;
    float scale_log2e;
    uint32_t q_flip; // set by the launch: sign bits to flip in pairs of query elements,
    int search;      // and whether the workgroups look for their tiles
};

// head_dim and dtype are checked by the caller; hipErrorInvalidValue where a launch would need
// 2^31 workgroups or more in a grid dimension.
hipError_t launch_kv_append(const AppendArgs &a, int head_dim, int dtype, hipStream_t st);
hipError_t launch_kv_evict(const EvictArgs &a, int head_dim, hipStream_t st);
size_t attn_cached_workspace(int n, int q_heads, int kv_heads, int head_dim, int q_len,
                             int max_len, bool weights);
hipError_t launch_attn_cached(const CachedArgs &a, int head_dim, int dtype, hipStream_t st);
hipError_t launch_attn_prompt(const PromptArgs &a, int head_dim, int dtype, hipStream_t st);

} // namespace mq
