// Attention over a paged cache: what its kernels share.
#pragma once

#include "h3qk_attn.cuh"
#include "h3qk_cache.cuh"

namespace h3qk_pages {

// A sequence's `n` query rows and the `group` heads that share a K/V head
// form n * group packed rows: packed row r is query row r / group, head
// kv * group + r % group.  So a tile of packed rows reads each key once for
// all of its heads, and a causal tile's rows stand close together.
struct Attn {
    Pool c;
    const int32_t* offsets;      // or null: `each` rows a sequence
    int32_t each, tokens, max_rows;
    int32_t heads, group, causal;
    float scale, cap;
    const float* slopes;
    const int32_t* prefix_lens;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_token, q_head, out_token, out_head;  // elements
    float* lse;                  // [heads][tokens]
    float* part;                 // partial results
    int64_t few;                 // sequences of at most so many packed rows go to the kernel for few rows
    int32_t least;               // few rows: units that a block takes at least
    int32_t tiles, parts;        // many rows: tiles of the longest sequence; blocks that share a tile's keys
    unsigned int* stuck;
};

// One sequence as the attention kernels see it.
struct Sequence {
    int first, n, keys, start, prefix;
};
__device__ __forceinline__ Sequence sequence_of(const Attn& p, int item)
{
    const Rows r = rows_of(p.offsets, p.each, p.tokens, item);
    Sequence s;
    s.first = r.first;
    s.n = min(r.n, p.max_rows);
    s.keys = keys_of(p.c, item);
    // (rows that max_rows hides are still the last ones of the cache)
    s.start = s.keys - r.n;
    s.prefix = p.prefix_lens ? max(__ldg(p.prefix_lens + item), 0) : 0;
    return s;
}
__device__ __forceinline__ int limit_of(const Sequence& s, bool causal, int i)
{
    return causal ? max(min(s.keys, max(s.prefix, s.start + i + 1)), 0) : s.keys;
}

__device__ __forceinline__ h3qk_core::Bend bend_of(const Attn& p, int head, float raw)
{
    // `raw`: what a raw score has to be multiplied with to be q.k.
    using namespace h3qk_core;
    Bend b;
    b.plain = p.scale * kLog2e * raw;
    b.in = p.cap > 0.0f ? fminf(p.scale * 2.0f * kLog2e / p.cap, 3.0e38f) * raw : b.plain;
    b.cap = p.cap * kLog2e;
    b.slope = p.slopes ? __ldg(p.slopes + head) * kLog2e : 0.0f;
    return b;
}

// Host side: the kernels' launchers.
constexpr int kUnit = 64;  // keys of a unit of work of the kernel for few rows
H3QK_HIDDEN int few_blocks(bool e2m1, int row_tile);
H3QK_HIDDEN int64_t few_floats(int blocks, int rows, int dim);
H3QK_HIDDEN cudaError_t cache_few(bool bf16, bool e2m1, int row_tile, int blocks, const Attn& p, cudaStream_t st);

}  // namespace h3qk_pages
