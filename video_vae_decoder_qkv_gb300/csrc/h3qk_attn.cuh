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
    float* part;              // partial results
    int32_t splits, chunk;    // few rows: keys per block
    int32_t tiles, whole, tail, parts;  // many rows: see TilePlan
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
// slope * distance, times log2(e).  With e = 2^(-2 |x| log2 e) and
// y = 1 + e in [1, 2], tanh |x| = (1 - e) / y and 1 - tanh^2 = 4 e / y^2, to an
// absolute 2^-21 (the hardware's own tanh has 2^-11).  Four scores share one
// hardware reciprocal, of the product of their y (1/x has half the rate of
// 2^x, 16 a cycle and SM, and would bound the capped kernels; a reciprocal
// from multiply-adds measured slower).
// Which bends a call has is fixed at compile time.  A NaN score makes all four
// NaN, so they have to be of one row; APART: the scores at even places belong to
// one row and those at odd places to another, and two share a reciprocal.
//
// The error is absolute in tanh, so a cap far above the scores costs them
// digits: cap 2^-21.  Beyond kWideCap, where that passes 2^-11 (fp16 rounds p
// to 2^-12), scores below a quarter of the cap take tanh's series instead, to
// a relative 2^-22.  That is an instance of its own: 16 heads of 4096 x 128,
// bf16, take 319 us forward and 777 backward with a cap of 2000, 184 and 559
// with one of 30.
enum Bends { kPlain = 0, kCapped = 1, kSloped = 2, kWide = 4 };
constexpr float kWideCap = 1024.0f;

struct Bend {
    float in;     // scale * 2 log2(e) / cap, or scale * log2(e) without a cap
    float plain;  // scale * log2(e)
    float cap;    // cap * log2(e)
    float slope;  // slope * log2(e)
};

__device__ __forceinline__ Bend bend_of(const Params& p, int head)
{
    Bend b;
    b.plain = p.scale * kLog2e;
    // (the smallest caps would make this infinite, and a score of 0 NaN)
    b.in = p.cap > 0.0f ? fminf(p.scale * 2.0f * kLog2e / p.cap, 3.0e38f) : b.plain;
    b.cap = p.cap * kLog2e;
    b.slope = p.slopes ? __ldg(p.slopes + head) * kLog2e : 0.0f;
    return b;
}

// tanh(u) / u for |u| < 1/4, given w = (2 u log2 e)^2, to 2^-26: 1 - u^2/3 +
// 2u^4/15 - 17u^6/315 + 62u^8/2835, tanh's Taylor series.  kSmall is the bound
// on |2 u log2 e|.
constexpr float kSmall = 0.72f;
constexpr float kHalfLn2Sq = 0.25f * kLn2 * kLn2;
__device__ __forceinline__ uint64_t tanh_series(uint64_t w)
{
    using namespace h3qk_tc;
    auto both = [](float v) { return pair(v, v); };
    const uint64_t t = mul_pair(w, both(kHalfLn2Sq));
    uint64_t p = fma_pair(t, both(62.0f / 2835.0f), both(-17.0f / 315.0f));
    p = fma_pair(t, p, both(2.0f / 15.0f));
    p = fma_pair(t, p, both(-1.0f / 3.0f));
    return fma_pair(t, p, both(1.0f));
}

// The exponents of four raw scores (two pairs) at distances far, far + dir,
// ...; with KEEP, also 1 - tanh^2 of a cap.
template <int BENDS, bool KEEP, bool APART = false>
__device__ __forceinline__ void bend_four(uint64_t (&z)[2], const Bend& b, float far, float dir, uint64_t (&keep)[2])
{
    using namespace h3qk_tc;
    const uint64_t in = pair(b.in, b.in);
    [[maybe_unused]] uint64_t flat[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (BENDS & kWide) flat[i] = mul_pair(z[i], pair(b.plain, b.plain));
        z[i] = mul_pair(z[i], in);
    }
    if constexpr (BENDS & kCapped) {
        const uint64_t one = pair(1.0f, 1.0f), cap = pair(b.cap, b.cap), less = pair(-b.cap, -b.cap);
        float lo[2], hi[2];
        uint64_t e[2], y[2], r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            unpair(lo[i], hi[i], z[i]);
            e[i] = pair(exp2_fast(-fabsf(lo[i])), exp2_fast(-fabsf(hi[i])));
            y[i] = add_pair(e[i], one);
        }
        float p_lo, p_hi;
        unpair(p_lo, p_hi, mul_pair(y[0], y[1]));
        uint64_t both;  // 1 / (y[0] y[1])
        if constexpr (APART) {
            both = pair(rcp_fast(p_lo), rcp_fast(p_hi));
        } else {
            const float all = rcp_fast(p_lo * p_hi);
            both = pair(all * p_hi, all * p_lo);
        }
        r[0] = mul_pair(both, y[1]);
        r[1] = mul_pair(both, y[0]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (KEEP) keep[i] = mul_pair(mul_pair(e[i], pair(4.0f, 4.0f)), mul_pair(r[i], r[i]));
            float t_lo, t_hi;
            unpair(t_lo, t_hi, mul_pair(fma_pair(e[i], less, cap), r[i]));
            t_lo = copysignf(t_lo, lo[i]);
            t_hi = copysignf(t_hi, hi[i]);
            if constexpr (BENDS & kWide) {
                const uint64_t both_in = pair(lo[i], hi[i]);
                float f_lo, f_hi;
                unpair(f_lo, f_hi, mul_pair(flat[i], tanh_series(mul_pair(both_in, both_in))));
                if (fabsf(lo[i]) < kSmall) t_lo = f_lo;
                if (fabsf(hi[i]) < kSmall) t_hi = f_hi;
            }
            z[i] = pair(t_lo, t_hi);
        }
    }
    if constexpr (BENDS & kSloped) {
        const uint64_t slope = pair(-b.slope, -b.slope);
        z[0] = fma_pair(pair(fabsf(far), fabsf(far + dir)), slope, z[0]);
        z[1] = fma_pair(pair(fabsf(far + 2.0f * dir), fabsf(far + 3.0f * dir)), slope, z[1]);
    }
}

// Registers a thread of the tile kernels' 12 warps: 168 at launch, which the 8
// warps of arithmetic and the 4 others then share out as 8 x 216 + 4 x 72 =
// 12 x 168.
constexpr int kLaunchRegs = 168, kMathRegs = 216, kOtherRegs = 72;

// Once per kernel and device: its shared memory limit.  A kernel that was
// launched with other than kLaunchRegs registers would wait for registers
// that do not exist: refused.
template <typename K>
cudaError_t ready(K* kernel, int smem, bool (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e == cudaSuccess && a.numRegs != kLaunchRegs) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    done[dev] = e == cudaSuccess;
    return e;
}

// Many rows: the blocks' tiles (256 query rows of a head) in one row, `tiles`
// a head.  A last round of tiles that would leave most SMs idle is cut along
// the keys: the first `whole` tiles have a block each, the `tail` ones after
// them `parts`, whose results a second kernel joins.
constexpr int kRowTile = 256;
struct TilePlan {
    int64_t tiles, whole, tail, parts;  // tail 0: nothing is cut
};
// Floats that a part leaves: per row O[dim], then m and sum of every row.
__host__ __device__ inline int64_t tile_part_floats(int dim) { return static_cast<int64_t>(kRowTile) * (dim + 2); }

// Host side: the kernels' launchers.
struct Maps {
    CUtensorMap q, k, v, dout;
};
// A tensor's map [items][heads][rows][dim]: boxes of box_rows by 64 channels,
// 128-byte swizzle, zeros past the ends.
H3QK_HIDDEN bool encode_map(CUtensorMap* m, const void* data, bool bf16, int64_t dim, int64_t rows, int64_t heads, int64_t items,
                            int64_t row_bytes, int64_t head_bytes, int64_t item_bytes, int box_rows);
// The current device's count of blocks that gave up waiting.
H3QK_HIDDEN unsigned int* stuck_addr();
// The runtime could not give the stuck counter or a tensor map.
H3QK_HIDDEN h3qk_status no_maps();
H3QK_HIDDEN cudaError_t forward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st);
H3QK_HIDDEN cudaError_t forward_split(bool bf16, const Params& p, cudaStream_t st);
H3QK_HIDDEN cudaError_t backward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st);

}  // namespace h3qk_core
