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

// What a block takes at least: for few rows units of 64 keys, two turns of its
// warps; for many, tiles of 128 keys, to be worth its start and the join.
constexpr int kLeastUnits = 4, kLeastTiles = 4;
// What a block of a cluster takes at most: beyond, the line's shares are shorter.
constexpr int kMostUnits = 16;

// Calls whose sequences have at most kFew packed rows go to the kernel for few
// rows, which reads (and converts) their keys once for 8 or 16 of them; others
// to the tiles of 256, of which even a row costs a whole softmax.  24 caches of
// up to 8,192 keys in 4 bits, 20 packed rows, capped scores: 69 us in two tiles
// of 16, 152 in tiles of 256.  A call that mixes long chunks with single tokens
// stays in one kernel, whose equal shares end together, and its tokens take
// tiles of 256.
constexpr int kFew = 32;

// How a call is cut, from its sizes alone.
struct Cut {
    bool tiles;            // the kernel for many rows
    int row_tile, blocks;  // few rows
    int cluster;           // their row tiles, where clusters take them
    TileGrid grid;         // many rows
    int64_t floats;        // of partial results
};
Cut cut_of(const h3qk_cache& c, const h3qk_cache_attn& a, int64_t max_rows)
{
    Cut t = {};
    const int64_t group = a.heads / c.kv_heads, packed = max_rows * group;
    const int sms = h3qk_internal_sm_count();
    t.tiles = packed > kFew;
    if (!t.tiles) {
        t.row_tile = packed <= 8 ? 8 : 16;
        const int64_t tiles = (packed + t.row_tile - 1) / t.row_tile;
        const int64_t per = (static_cast<int64_t>(c.max_pages) * c.page_size + kUnit - 1) / kUnit;
        const double units = static_cast<double>(c.batch) * c.kv_heads * tiles * (per > 0 ? per : 1);
        const int most = few_blocks(c.format == H3QK_E2M1, t.row_tile);
        // A cluster a run, while all of them fit the GPU at once and a block's
        // share of the longest cache stays short.
        const double clustered = static_cast<double>(c.batch) * c.kv_heads * tiles * kCluster;
        if (clustered <= most && per <= kCluster * kMostUnits) {
            t.cluster = static_cast<int>(tiles);
            t.blocks = static_cast<int>(clustered);
            return t;
        }
        const double want = std::ceil(units / kLeastUnits);
        t.blocks = want < most ? static_cast<int>(want) : most;
        t.floats = few_floats(t.blocks, t.row_tile, c.head_dim);
    }
    if (t.tiles) {
        // Tiles of 256 at most: of all rows in full ones, and a partial one a sequence; or of sequences as long as may be.
        const double by_rows = std::floor(static_cast<double>(a.tokens) * group / h3qk_core::kRowTile) + c.batch;
        const double by_batch = std::ceil(static_cast<double>(packed) / h3qk_core::kRowTile) * c.batch;
        const double keys = std::ceil(static_cast<double>(c.max_pages) * c.page_size / 128);
        const double units = (by_rows < by_batch ? by_rows : by_batch) * c.kv_heads * (keys > 1 ? keys : 1);
        const double want = std::ceil(units / kLeastTiles);
        t.grid.blocks = want < sms ? static_cast<int>(want) : sms;
        t.floats = t.grid.blocks == 1 ? 0 : t.grid.blocks * (2 * tile_floats(c.head_dim) + kBrokenFloats);
    }
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
    // packed rows to full tiles, all heads' rows, and the join's grid fit 31 bits
    if (*rows * (a.heads / c.kv_heads) > INT32_MAX + INT64_C(1) - h3qk_core::kRowTile) return H3QK_ERR_INVALID_ARG;
    if (a.tokens * a.heads > INT32_MAX || static_cast<double>(a.heads) * c.batch * kFew > INT32_MAX) return H3QK_ERR_INVALID_ARG;
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
    const Cut cut = cut_of(*cache, *call, rows);
    return static_cast<size_t>(cut.floats) * 4;
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
    p.bf16 = a.dtype == H3QK_BF16;
    p.scale = a.scale > 0.0f ? a.scale : 1.0f / std::sqrt(static_cast<float>(c.head_dim));
    p.cap = a.softcap;
    p.slopes = a.slopes;
    p.prefix_lens = a.prefix_lens;
    p.q = static_cast<const uint16_t*>(a.q);
    p.out = static_cast<uint16_t*>(a.out);
    p.q_token = a.q_token_stride, p.q_head = a.q_head_stride;
    p.out_token = a.out_token_stride, p.out_head = a.out_head_stride;
    p.lse = a.lse;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = p.bf16 != 0, e2m1 = c.format == H3QK_E2M1;
    p.part = static_cast<float*>(a.workspace);
    cudaError_t e;
    if (!cut.tiles) {
        p.least = kLeastUnits;
        p.cluster = cut.cluster;
        e = cache_few(e2m1, cut.row_tile, cut.blocks, p, st);
    } else {
        p.least = kLeastTiles;
        p.stuck = h3qk_core::stuck_addr();
        Maps m = {};
        bool ok = p.stuck != nullptr;
        if (!e2m1) {
            // A pool without pages is described as its rows' own tensor: no page of it is ever named.
            const bool none = c.pages == 0;
            const int64_t row = c.head_dim * 2, rows_a_page = none ? 16 : c.page_size;
            const int box = static_cast<int>(c.page_size < 128 ? c.page_size : 128);
            const void* data[2] = {none ? a.q : c.k, none ? a.q : c.v};
            CUtensorMap* maps[2] = {&m.k, &m.v};
            const int64_t strides[2][3] = {{p.c.k_row, p.c.k_head, p.c.k_page}, {p.c.v_row, p.c.v_head, p.c.v_page}};
            for (int i = 0; i < 2; ++i)
                ok = ok && h3qk_core::encode_map(maps[i], data[i], bf16, c.head_dim, rows_a_page, none ? 1 : c.kv_heads,
                                                 none ? 1 : c.pages, none ? row : strides[i][0], none ? 16 * row : strides[i][1],
                                                 none ? 16 * row : strides[i][2], box);
        }
        if (!ok) return h3qk_core::no_maps();
        if (e2m1) e = bf16 ? cache_tiles_e2m1_bf16(p, m, cut.grid, st) : cache_tiles_e2m1_fp16(p, m, cut.grid, st);
        else e = bf16 ? cache_tiles_bf16(p, m, cut.grid, st) : cache_tiles_fp16(p, m, cut.grid, st);
    }
    return h3qk_ops::status_of(e);
}
