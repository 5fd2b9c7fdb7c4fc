// What the attention kernels share: the call's parameters, the stretch of
// rows a block works on, and the score's bend (cap, distance).
//
// Every mask of the operator shows row i a prefix of its stretch's keys:
// keys j < min(keys, max(prefix, start + i + 1)) when causal, all `keys`
// otherwise.  A document is a stretch of its own, and blocks never span two,
// so masking one score is a single comparison, tiles beyond the last visible
// key are never loaded, and nothing of one document is ever multiplied into
// another's rows.
#pragma once

#include "h3qk_ops.cuh"
#include "h3qk_tc.cuh"

namespace h3qk_core {

struct Strides {
    int64_t item, head, row;  // elements
};

struct Params {
    int32_t batch, heads, kv_heads, group, dim;
    int32_t q_rows, kv_rows;  // rows of the tensors
    int32_t causal, docs;
    float scale, cap;         // cap 0: none
    const float* slopes;
    const int32_t *prefix_lens, *doc_offsets, *q_lens, *kv_lens, *q_starts;
    const uint16_t *q, *k, *v;
    Strides qs, ks, vs;
    uint16_t* out;
    Strides os;
    float* lse;               // [batch][heads][q_rows]
    const uint16_t* dout;     // backward
    Strides dos;
    uint16_t *dq, *dk, *dv;
    Strides dqs, dks, dvs;
    float* delta;             // [batch][heads][q_rows]
    float* part;              // split: partial results
    int32_t splits, chunk;    // split: keys per block
    unsigned int* stuck;      // counts blocks whose waits ran out
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kFar = 1 << 30;  // lengths and positions stay below this

struct Stretch {
    int item;
    int row0;    // first row in the q tensor (documents: also in the k tensor)
    int k0;      // first key row in the k tensor
    int span;    // rows to write (those past `rows` get zeros)
    int rows;    // rows that attend
    int keys;
    int start;   // position of row 0 among the keys
    int prefix;
    int tile;    // this block's tile within the stretch
};

__device__ __forceinline__ int clamp_len(int v, int most) { return min(max(v, 0), most); }

// Keys that row i sees.
__device__ __forceinline__ int limit_of(const Stretch& s, bool causal, int i)
{
    return causal ? min(s.keys, max(s.prefix, s.start + i + 1)) : s.keys;
}

// The stretch and tile (of `size` rows; of keys with `by_keys`) of block
// number `block` along the grid; false past the last one.  Documents: each
// one's tiles follow the last one's, found by a warp-wide running sum over
// the offsets; the rows after the last document are a stretch without keys.
__device__ __forceinline__ bool find_stretch(Stretch& s, const Params& p, int block, int item, int size, bool by_keys)
{
    const int most_q = p.q_rows, most_k = p.kv_rows;
    if (p.docs == 0) {
        s.item = item;
        s.row0 = s.k0 = 0;
        s.tile = block;
        s.keys = p.kv_lens ? clamp_len(__ldg(p.kv_lens + item), most_k) : most_k;
        s.rows = p.q_lens ? clamp_len(__ldg(p.q_lens + item), most_q) : most_q;
        s.span = by_keys ? most_k : most_q;
        s.prefix = p.prefix_lens ? clamp_len(__ldg(p.prefix_lens + item), kFar) : 0;
        s.start = p.q_starts ? min(max(__ldg(p.q_starts + item), -kFar), kFar) : (most_q == most_k ? 0 : s.keys - s.rows);
        return static_cast<int64_t>(block) * size < s.span;
    }
    s.item = 0;
    s.start = 0;
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int d0 = 0; d0 <= p.docs; d0 += 32) {
        const int d = d0 + lane;
        int lo = 0, hi = 0;
        if (d <= p.docs) {
            lo = d == 0 ? 0 : clamp_len(__ldg(p.doc_offsets + d), most_q);
            hi = d == p.docs ? most_q : clamp_len(__ldg(p.doc_offsets + d + 1), most_q);
        }
        const int len = max(hi - lo, 0);
        const int tiles = (len + size - 1) / size;
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const bool here = block >= before + sum - tiles && block < before + sum;
        const unsigned vote = __ballot_sync(0xffffffffu, here);
        if (vote) {
            const int src = __ffs(vote) - 1;
            s.row0 = s.k0 = __shfl_sync(0xffffffffu, lo, src);
            s.span = __shfl_sync(0xffffffffu, len, src);
            s.tile = block - __shfl_sync(0xffffffffu, before + sum - tiles, src);
            const bool tail = d0 + src == p.docs;
            s.rows = s.keys = tail ? 0 : s.span;
            s.prefix = p.prefix_lens && !tail ? clamp_len(__ldg(p.prefix_lens + d0 + src), kFar) : 0;
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return false;
}

// Blocks along the grid that cover every stretch.
inline int64_t tiles_of(const Params& p, int64_t rows, int size)
{
    return (rows + size - 1) / size + (p.docs ? p.docs : 0);
}

// A raw score q.k as a power of two's exponent: cap * tanh(scale q.k / cap) -
// slope * distance, times log2(e).  With e = 2^(-2 |x| log2 e),
// tanh |x| = (1 - e) / (1 + e) and 1 - tanh^2 = 4 e / (1 + e)^2, to an
// absolute 2^-20 (the hardware's own tanh has 2^-11).  The reciprocal of
// y = 1 + e in [1, 2] is made of multiply-adds, two at a time: the hardware's
// 1/x runs at half the rate of its 2^x and would bound the capped kernels.
// p(y) = (1 - T3(2y - 3) / T3(-3)) / y, a polynomial of degree 2 with
// |1 - y p| <= 1/99 on [1, 2] (T3: Chebyshev's), then p (1 + h + h^2) with
// h = 1 - y p, which leaves h^3, about 2^-20.
// Which bends a call has is fixed at compile time.
enum Bends { kPlain = 0, kCapped = 1, kSloped = 2 };

struct Bend {
    float in;     // scale * 2 log2(e) / cap, or scale * log2(e) without a cap
    float cap;    // cap * log2(e)
    float slope;  // slope * log2(e)
};

__device__ __forceinline__ Bend bend_of(const Params& p, int head)
{
    Bend b;
    b.in = p.cap > 0.0f ? p.scale * 2.0f * kLog2e / p.cap : p.scale * kLog2e;
    b.cap = p.cap * kLog2e;
    b.slope = p.slopes ? __ldg(p.slopes + head) * kLog2e : 0.0f;
    return b;
}

// The exponent of a pair of raw scores whose keys are `far` away; with
// `keep`, also 1 - tanh^2 of a cap.
template <int BENDS, bool KEEP>
__device__ __forceinline__ uint64_t bend_pair(uint64_t z, const Bend& b, float far_lo, float far_hi, uint64_t* keep)
{
    using namespace h3qk_tc;
    z = mul_pair(z, pair(b.in, b.in));
    if constexpr (BENDS & kCapped) {
        const uint64_t one = pair(1.0f, 1.0f);
        float lo, hi;
        unpair(lo, hi, z);
        const uint64_t e = pair(exp2_fast(-fabsf(lo)), exp2_fast(-fabsf(hi)));
        const uint64_t y = fma_pair(e, pair(-1.0f, -1.0f), pair(-1.0f, -1.0f));  // -(1 + e)
        uint64_t r = fma_pair(fma_pair(y, pair(32.0f / 99.0f, 32.0f / 99.0f), pair(144.0f / 99.0f, 144.0f / 99.0f)), y,
                              pair(210.0f / 99.0f, 210.0f / 99.0f));
        const uint64_t h = fma_pair(y, r, one);
        r = fma_pair(r, fma_pair(h, h, h), r);
        if constexpr (KEEP) *keep = mul_pair(mul_pair(e, pair(4.0f, 4.0f)), mul_pair(r, r));
        float t_lo, t_hi;
        unpair(t_lo, t_hi, mul_pair(fma_pair(e, pair(-b.cap, -b.cap), pair(b.cap, b.cap)), r));
        z = pair(copysignf(t_lo, lo), copysignf(t_hi, hi));
    }
    if constexpr (BENDS & kSloped) z = fma_pair(pair(fabsf(far_lo), fabsf(far_hi)), pair(-b.slope, -b.slope), z);
    return z;
}

// Host side: the kernels' launchers.
struct Maps {
    CUtensorMap q, k, v, dout;
};
H3QK_HIDDEN cudaError_t forward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st);
H3QK_HIDDEN cudaError_t forward_split(bool bf16, const Params& p, cudaStream_t st);
H3QK_HIDDEN cudaError_t backward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st);

}  // namespace h3qk_core
