// Host side of attention over a paged cache: argument checks and the choice
// of kernels.
#include <cmath>

#include "h3qk_cache_attn.cuh"
#include "h3qk_cache_host.h"

namespace {

using namespace h3qk_pages;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

constexpr int kLeastUnits = 4;

// How a call is cut, from its sizes alone.
struct Cut {
    int row_tile, blocks;  // few rows
    int64_t floats;        // of partial results
};
Cut cut_of(const h3qk_cache& c, const h3qk_cache_attn& a, int64_t max_rows)
{
    Cut t = {};
    const int64_t packed = max_rows * (a.heads / c.kv_heads);
    t.row_tile = packed <= 8 ? 8 : 16;
    const int64_t tiles = (packed + t.row_tile - 1) / t.row_tile;
    const int64_t per = (static_cast<int64_t>(c.max_pages) * c.page_size + kUnit - 1) / kUnit;
    const double units = static_cast<double>(c.batch) * c.kv_heads * tiles * (per > 0 ? per : 1);
    const int most = few_blocks(c.format == H3QK_E2M1, t.row_tile);
    const double want = std::ceil(units / kLeastUnits);
    t.blocks = want < most ? static_cast<int>(want) : most;
    t.floats = few_floats(t.blocks, t.row_tile, c.head_dim);
    return t;
}

// Sizes and options; `rows`: the most rows that a sequence may have.
h3qk_status check_call(const h3qk_cache& c, const h3qk_cache_attn& a, int64_t* rows)
{
    if (a.dtype != H3QK_FP16 && a.dtype != H3QK_BF16) return H3QK_ERR_INVALID_ARG;
    if (c.format != H3QK_E2M1 && c.format != a.dtype) return H3QK_ERR_INVALID_ARG;
    if (c.kv_heads < 1 || c.batch < 1 || a.heads < 1 || a.heads > 65535 || a.heads % c.kv_heads) return H3QK_ERR_INVALID_ARG;
    if (a.causal != 0 && a.causal != 1) return H3QK_ERR_INVALID_ARG;
    if (a.prefix_lens && !a.causal) return H3QK_ERR_INVALID_ARG;
    if (!(a.scale >= 0.0f) || !std::isfinite(a.scale)) return H3QK_ERR_INVALID_ARG;
    if (!(a.softcap >= 0.0f) || !std::isfinite(a.softcap)) return H3QK_ERR_INVALID_ARG;
    if (a.tokens < 0 || a.tokens >= (INT64_C(1) << 30) || a.max_rows < 0) return H3QK_ERR_INVALID_ARG;
    if (!a.q_offsets && a.tokens % c.batch) return H3QK_ERR_INVALID_ARG;
    *rows = a.q_offsets ? a.tokens : a.tokens / c.batch;
    if (a.max_rows > 0 && a.max_rows < *rows) *rows = a.max_rows;
    // the join's grid
    if (static_cast<double>(*rows) * a.heads * c.batch > 2e9) return H3QK_ERR_INVALID_ARG;
    return H3QK_OK;
}

h3qk_status check_rows(const void* data, int64_t token, int64_t head, const h3qk_cache& c, const h3qk_cache_attn& a, Range* r)
{
    if (!data) return H3QK_ERR_INVALID_ARG;
    const int64_t most = INT64_C(1) << 38;
    if (a.heads == 1) head = c.head_dim;
    if (a.tokens == 1) token = a.heads * head;
    if (token <= 0 || head <= 0 || token >= most || head >= most) return H3QK_ERR_INVALID_ARG;
    if (head < c.head_dim && a.heads > 1) return H3QK_ERR_INVALID_ARG;
    if (token < c.head_dim && a.tokens > 1) return H3QK_ERR_INVALID_ARG;
    if (token % 8 || head % 8 || !aligned(data, 16)) return H3QK_ERR_MISALIGNED;
    const double span = static_cast<double>(a.tokens) * token + static_cast<double>(a.heads) * head;
    if (span > 1e15) return H3QK_ERR_INVALID_ARG;
    *r = range_of(data, ((a.tokens - 1) * token + (a.heads - 1) * head + c.head_dim) * 2);
    return H3QK_OK;
}

}  // namespace

extern "C" size_t h3qk_cache_attention_workspace_bytes(const h3qk_cache* cache, const h3qk_cache_attn* call)
{
    int64_t rows;
    if (!cache || !call || check_call(*cache, *call, &rows) != H3QK_OK || rows == 0) return 0;
    return static_cast<size_t>(cut_of(*cache, *call, rows).floats) * 4;
}

extern "C" h3qk_status h3qk_cache_attention(const h3qk_cache* cache, const h3qk_cache_attn* call, h3qk_stream_t stream)
{
    Attn p = {};
    PoolRanges pool;
    h3qk_status s = check_pool(cache, false, &p.c, &pool);
    if (s != H3QK_OK) return s;
    if (!call) return H3QK_ERR_INVALID_ARG;
    const h3qk_cache& c = *cache;
    const h3qk_cache_attn& a = *call;
    int64_t rows;
    if ((s = check_call(c, a, &rows)) != H3QK_OK) return s;
    if (a.tokens == 0) return H3QK_OK;
    Range q, out;
    if ((s = check_rows(a.q, a.q_token_stride, a.q_head_stride, c, a, &q)) != H3QK_OK) return s;
    if ((s = check_rows(a.out, a.out_token_stride, a.out_head_stride, c, a, &out)) != H3QK_OK) return s;
    // rows of out may not run into one another
    const int64_t inner = a.heads > 1 && a.tokens > 1 ? (a.out_token_stride < a.out_head_stride ? a.tokens : a.heads) : 1;
    if (inner > 1) {
        const int64_t small = a.out_token_stride < a.out_head_stride ? a.out_token_stride : a.out_head_stride;
        const int64_t large = a.out_token_stride < a.out_head_stride ? a.out_head_stride : a.out_token_stride;
        if (large < (inner - 1) * small + c.head_dim) return H3QK_ERR_ALIAS;
    }
    if (!a.lse) return H3QK_ERR_INVALID_ARG;
    if (!aligned(a.lse, 4) || !aligned(a.slopes, 4) || !aligned(a.prefix_lens, 4) || !aligned(a.q_offsets, 4))
        return H3QK_ERR_MISALIGNED;
    const Cut cut = cut_of(c, a, rows);
    const size_t need = static_cast<size_t>(cut.floats) * 4;
    if (need && (!a.workspace || a.workspace_bytes < need)) return H3QK_ERR_INVALID_ARG;
    if (need && !aligned(a.workspace, 16)) return H3QK_ERR_MISALIGNED;
    const Range outs[3] = {out, range_of(a.lse, a.heads * a.tokens * 4), range_of(a.workspace, need)};
    const Range ins[10] = {q, pool.data[0], pool.data[1], pool.data[2], pool.data[3], pool.lists[0], pool.lists[1],
                           range_of(a.slopes, a.slopes ? a.heads * 4 : 0),
                           range_of(a.prefix_lens, a.prefix_lens ? c.batch * 4 : 0),
                           range_of(a.q_offsets, a.q_offsets ? (c.batch + 1) * 4 : 0)};
    for (int i = 0; i < 3; ++i) {
        for (int k = i + 1; k < 3; ++k)
            if (overlap(outs[i], outs[k])) return H3QK_ERR_ALIAS;
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return H3QK_ERR_ALIAS;
    }
    p.offsets = a.q_offsets;
    p.each = a.q_offsets ? 0 : static_cast<int32_t>(a.tokens / c.batch);
    p.tokens = static_cast<int32_t>(a.tokens);
    p.max_rows = static_cast<int32_t>(rows);
    p.heads = a.heads;
    p.group = a.heads / c.kv_heads;
    p.causal = a.causal;
    p.scale = a.scale > 0.0f ? a.scale : 1.0f / std::sqrt(static_cast<float>(c.head_dim));
    p.cap = a.softcap;
    p.slopes = a.slopes;
    p.prefix_lens = a.prefix_lens;
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = static_cast<uint16_t*>(a.out);
    p.q_token = a.q_token_stride, p.q_head = a.q_head_stride;
    p.out_token = a.out_token_stride, p.out_head = a.out_head_stride;
    p.lse = a.lse;
    p.part = static_cast<float*>(a.workspace);
    p.few = INT64_MAX;
    p.least = kLeastUnits;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return h3qk_ops::status_of(cache_few(a.dtype == H3QK_BF16, c.format == H3QK_E2M1, cut.row_tile, cut.blocks, p, st));
}
