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
    int32_t bf16;                // what q and out are
    float scale, cap;
    const float* slopes;
    const int32_t* prefix_lens;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_token, q_head, out_token, out_head;  // elements
    float* lse;                  // [heads][tokens]
    float* part;                 // partial results of the kernel that is launched
    int32_t least;               // units that a block takes at least
    int32_t cluster;             // few rows: 0, or row tiles of the longest sequence, a cluster a run
    unsigned int* stuck;
};

// Packed rows fit 31 bits; their division is the unsigned one, which is short.
__device__ __forceinline__ int divide(int a, int b) { return static_cast<int>(static_cast<unsigned>(a) / static_cast<unsigned>(b)); }

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
    // The length as it is given, beyond the table too, says where the rows stand
    // (those that max_rows hides among them).  start + i stays below it.
    s.start = max(__ldg(p.c.kv_lens + item), 0) - r.n;
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
    // (positive and finite, so that it keeps a hidden score's -infinity)
    b.plain = fminf(fmaxf(p.scale * kLog2e * raw, 0x1p-126f), 3.0e38f);
    // (finite before and after: an infinite factor would make a score of 0 NaN)
    b.in = p.cap > 0.0f ? fminf(fminf(p.scale * 2.0f * kLog2e / p.cap, 3.0e38f) * raw, 3.0e38f) : b.plain;
    b.cap = p.cap * kLog2e;
    b.slope = p.slopes ? __ldg(p.slopes + head) * kLog2e : 0.0f;
    return b;
}

// A row of bfloat16 becomes one of binary16: times 2^(141 - e), e the exponent
// field of its largest magnitude (given as bits), so that this comes to lie in
// [2^14, 2^15).  bfloat16's 8 digits fit down to 2^-17 there; below, a channel is
// off by up to 2^-25, which is 2^-39 of the row's largest magnitude.  That is more
// than binary32 sums lose only where the large channels meet zeros.  Rows with
// an infinity or NaN stay as they are.
__device__ __forceinline__ float raise_of(uint32_t top, int& e)
{
    e = top >> 7;
    e = e == 255 ? 141 : max(e, 15);
    return __int_as_float((127 + 141 - e) << 23);
}

// Writes 4 channels of one joined packed row (d = 0: its lse too).
__device__ __forceinline__ void finish_row(const Attn& p, const Sequence& s, int kv, int r, int d, float4 v, float top,
                                           float sum, float shift, float v_scale)
{
    using h3qk_tc::round_pair;
    const int i = divide(r, p.group), head = kv * p.group + r - i * p.group;
    const int64_t token = s.first + i;
    const float inv = sum == 0.0f ? 0.0f : v_scale / sum;
    if (d < p.c.dim) {
        uint2 w;
        w.x = p.bf16 ? round_pair<true>(v.x * inv, v.y * inv) : round_pair<false>(v.x * inv, v.y * inv);
        w.y = p.bf16 ? round_pair<true>(v.z * inv, v.w * inv) : round_pair<false>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(p.out + token * p.out_token + head * p.out_head + d) = w;
    }
    if (d == 0)
        p.lse[static_cast<int64_t>(head) * p.tokens + token] =
            sum == 0.0f ? -INFINITY : (top - shift + log2f(sum)) * h3qk_core::kLn2;
}

// Host side: the kernels' launchers.
struct Maps {
    CUtensorMap k, v;  // 16-bit pages
};
struct TileGrid {
    int blocks;
};
// Floats of a partial tile (per packed row O[dim], then m and sum), of which a
// block leaves two at most; and of the words that tell the join of them.
inline int64_t tile_floats(int dim) { return h3qk_core::tile_part_floats(dim); }
constexpr int kBrokenFloats = 5;
constexpr int kUnit = 64;    // keys of a unit of work of the kernel for few rows
constexpr int kCluster = 8;  // blocks that share a run without a second launch
H3QK_HIDDEN int few_blocks(bool e2m1, int row_tile);
H3QK_HIDDEN int64_t few_floats(int blocks, int rows, int dim);
H3QK_HIDDEN cudaError_t cache_few(bool e2m1, int row_tile, int blocks, const Attn& p, cudaStream_t st);
H3QK_HIDDEN cudaError_t cache_tiles_e2m1_fp16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st);
H3QK_HIDDEN cudaError_t cache_tiles_e2m1_bf16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st);
H3QK_HIDDEN cudaError_t cache_tiles_fp16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st);
H3QK_HIDDEN cudaError_t cache_tiles_bf16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st);

}  // namespace h3qk_pages
