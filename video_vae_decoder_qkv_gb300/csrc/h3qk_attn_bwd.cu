// Attention backward.  With p = 2^(s - lse) recomputed from the scores,
//   delta = sum_d dout out,  dp = dout v^T,  ds = p (dp - delta) bend'(z),
//   dv = p^T dout,  dq = scale ds k,  dk = scale ds^T q.
//
// Two kernels, each of which owns its sums: one block per 128 query rows for
// dq (and delta), one per 128 keys of a K/V head for dk and dv, which walks
// the query tiles of every head that shares them.  s and dp are computed
// twice (7 products instead of 5), which buys results without atomics, the
// same bits every time, and no binary32 copy of dq in memory.
//
// 40 heads of 8160 x 8160 x 128, bf16: dq 1.25 ms, dk and dv 1.53 ms: the
// tensor unit bounds both, at 1.63 and 1.78 PFLOP/s of products run (1.23 of
// the 10 D a pair that the gradient needs).  32 heads of 8192 x 8192 x 64,
// fp16: 0.76 and 0.92 ms; there the arithmetic takes longer (about 1,000 and
// 1,300 cycles a tile of 128 x 128 against 768 and 1,024 of products), mostly
// in waits: counters show the tensor unit at 44 and 49 %, 2^x at 29 and 26 %.
// Twice as many warps on the same arithmetic measured 7 % slower.
//
// Both keep scores and dp in TMEM with the block's own rows as lanes, eight
// warps turn them into p and ds (one thread a row and half the columns), and
// p and ds return to TMEM as 16-bit A operands over the columns they came
// from, each half of the warps within its own columns.  The tensor unit works
// in order, so a product may be issued behind the one that still reads its
// destination's old contents.
#include "h3qk_attn.cuh"

#include <type_traits>

namespace {

using namespace h3qk_tc;
using h3qk_core::Bend;
using h3qk_core::Params;
using h3qk_core::Stretch;

constexpr int kTile = 128;
constexpr int kThreads = 384;           // 8 warps of arithmetic; products, loads, row statistics
constexpr int kBlockBytes = 128 * 128;  // 64 columns of a tile

template <int DP>
struct BwdShape {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kTiles = (2 + kStages) * kTileBytes;  // the barriers follow
};

struct BwdShared {
    uint64_t full[8], empty[8];
    uint64_t own, fixed[2], done, drain;
    uint64_t s_full[2], s_free[2], dp_full[2], p_ready[2], ds_ready[2], st_full[2], st_empty[2];
    uint32_t tmem;
    int stop;
    alignas(16) float lse[2][kTile];  // (dq: how far out's rounding moves delta)
    alignas(16) float delta[2][kTile];
};

// P is kept 2^10 larger in fp16, so that flat rows over many keys do not fall
// into subnormals (p <= 1, so 2^10 is far from overflow); dv takes it back.
template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 10.0f;
template <bool BF16>
constexpr float kDrop = BF16 ? 1.0f : 1.0f / 1024.0f;

// A rounding to the type: relative, and absolute among fp16's smallest numbers.
template <bool BF16>
constexpr float kRound = BF16 ? 1.0f / 256.0f : 1.0f / 2048.0f;
template <bool BF16>
constexpr float kTiny = BF16 ? 0.0f : 1.0f / 33554432.0f;

// What a block whose waits ran out leaves in its rows (by way of delta, also in
// the gradients of the keys that they see).
__device__ __forceinline__ float given_up() { return __int_as_float(0x7fc00000); }

// The tile, head and item of a block.  The grid is [tiles][heads][items], so a
// head's tiles follow one another and its streamed rows stay in L2.  Causal
// tiles are of unequal length: the longest of all heads (late rows, early keys)
// go first.
struct Place3 {
    int tile, head, item;
};
__device__ __forceinline__ Place3 place_of(bool causal, bool late_first, int heads, int items)
{
    if (!causal) return Place3{static_cast<int>(blockIdx.x), static_cast<int>(blockIdx.y), static_cast<int>(blockIdx.z)};
    const int tiles = gridDim.x;
    int64_t t = (static_cast<int64_t>(blockIdx.z) * heads + blockIdx.y) * tiles + blockIdx.x;
    Place3 at;
    at.head = static_cast<int>(t % heads);
    t /= heads;
    at.item = static_cast<int>(t % items);
    at.tile = static_cast<int>(t / items);
    if (late_first) at.tile = tiles - 1 - at.tile;
    return at;
}

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int blocks, int row, int head, int item,
                                          uint32_t bar)
{
    for (int b = 0; b < blocks; ++b) tma_load(dst + b * kBlockBytes, map, 64 * b, row, head, item, bar);
}

// Clears rows [first, 128) of a tile (one warp).
__device__ __forceinline__ void clear_rows(uint32_t tile, int blocks, int first)
{
    const int lane = threadIdx.x & 31;
    for (int b = 0; b < blocks; ++b)
        for (int o = first * 128 + lane * 16; o < kBlockBytes; o += 512)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * kBlockBytes + o), "r"(0) : "memory");
}

// a b^T over the channels: both tiles K-major.  `then` gets an arrival when
// the product is done.
template <int DP>
__device__ __forceinline__ void product_rows(uint32_t d, uint32_t a_tile, uint32_t b_tile, int steps, uint32_t shape,
                                             uint32_t then)
{
    const uint64_t a = tile_desc(a_tile, 16), b = tile_desc(b_tile, 16);
    if (elect_lane()) {
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
            if (i < steps) {
                const uint32_t off = ((i >> 2) * kBlockBytes + (i & 3) * 32) >> 4;
                mma_ss(d, a + off, b + off, shape, i > 0);
            }
        mma_commit(then);
    }
    __syncwarp();
}

// d += a b over 128 rows of b: a 16-bit pairs in TMEM, its two halves 64
// columns apart; b with its channels as N.
__device__ __forceinline__ void product_sum(uint32_t d, uint32_t a, uint32_t b_tile, uint32_t shape, bool add, uint32_t then)
{
    const uint64_t b = tile_desc(b_tile, kBlockBytes);
    if (elect_lane()) {
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
            mma_ts(d, a + (i >> 2) * 64 + (i & 3) * 8, b + (i * 2048 >> 4), shape, add || i > 0);
        mma_commit(then);
    }
    __syncwarp();
}

__device__ __forceinline__ void signal(uint32_t bar)
{
    if (elect_lane()) mma_commit(bar);
    __syncwarp();
}

// Writes DP/2 (or DP) columns of TMEM, scaled and rounded, as part of a row.
template <bool BF16, int COLS>
__device__ __forceinline__ void write_row(uint16_t* dst, uint32_t cols, int first, int dim, float by, bool zero, bool write)
{
#pragma unroll
    for (int d = 0; d < COLS; d += 32) {
        uint32_t o[32];
        tmem_ld32(o, cols + d);
        tmem_wait_ld(o);
        if (write) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (first + d + 8 * q < dim) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = zero ? 0u
                                    : round_pair<BF16>(__uint_as_float(o[8 * q + 2 * e]) * by,
                                                       __uint_as_float(o[8 * q + 2 * e + 1]) * by);
                    *reinterpret_cast<uint4*>(dst + first + d + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
    }
}

// Given up: loads in flight must land before the block leaves.
__device__ __forceinline__ void drain_loads(uint32_t full, int stages, int issued)
{
    for (int i = max(0, issued - stages); i < issued; ++i)
        for (int t = 0; t < kMaxTries && !bar_test(full + 8 * (i % stages), (i / stages) & 1); ++t) {}
}

__device__ __forceinline__ void drain_products(uint32_t bar)
{
    mma_commit(bar);
    for (int t = 0; t < kMaxTries && !bar_test(bar, 0); ++t) {}
}

// ---------------------------------------------------------------------------
// dq: a block's 128 query rows against the keys they see.  S and dP take
// three buffers of 128 columns.  Up to 64 channels the arithmetic bounds the
// kernel, and it should always find its next operand done:
//   tensor unit   S0 dP0 S1 | dP1 dQ0 S2 | dP2 dQ1 S3 | ...
// dP of the next tile goes where S of this one was as soon as all warps have
// it in registers, and the S after that where ds was once dQ has read it.
// Beyond, the tensor unit bounds it, and fetching V a turn earlier only takes
// room in the ring from the loads (12 % slower); there S alone is ahead:
//   tensor unit   S0 dP0 | S1 dQ0 dP1 | S2 dQ1 dP2 | ...
// ---------------------------------------------------------------------------
template <bool BF16, int DP, int BENDS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                        const __grid_constant__ Params p)
{
    using Shape = BwdShape<DP>;
    constexpr int kStages = Shape::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    BwdShared& sh = *reinterpret_cast<BwdShared*>(smem_raw + Shape::kTiles);
    const uint32_t base = smem_addr(smem_raw);
    if (base & 1023u) {  // the swizzle needs it; the launch gives it
        if (threadIdx.x == 0) atomicAdd(p.stuck, 1u);
        return;
    }
    const uint32_t q_smem = base, do_smem = base + Shape::kTileBytes, ring = base + 2 * Shape::kTileBytes;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const Place3 block = place_of(p.causal, true, p.heads, p.batch);
    const int head = block.head, kv_head = head / p.group;

    Stretch s;
    if (!h3qk_core::find_stretch(s, p, block.tile, block.item, kTile, false)) return;
    const int tile_row = s.tile * kTile;
    const int last = min(tile_row + kTile, s.rows) - 1;
    const int seen = last < tile_row ? 0 : max(h3qk_core::limit_of(s, p.causal, last), 0);
    const int n = (seen + kTile - 1) / kTile;
    const bool fix = n * kTile > seen && s.k0 + seen < p.kv_rows;

    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty), own = smem_addr(&sh.own);
    const uint32_t s_full = smem_addr(sh.s_full), s_free = smem_addr(sh.s_free), dp_full = smem_addr(sh.dp_full);
    const uint32_t ds_ready = smem_addr(sh.ds_ready);
    const uint32_t fixed = smem_addr(sh.fixed), done = smem_addr(&sh.done);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, 1);
            bar_init(empty + 8 * i, 1);
        }
        bar_init(own, 1);
        for (int i = 0; i < 2; ++i) bar_init(fixed + 8 * i, 1);
        bar_init(done, 1);
        bar_init(smem_addr(&sh.drain), 1);
        // Two of each, taken in turn: neither side can be two turns ahead.
        for (int i = 0; i < 2; ++i) {
            bar_init(s_full + 8 * i, 1);
            bar_init(dp_full + 8 * i, 1);
            bar_init(s_free + 8 * i, 8);
            bar_init(ds_ready + 8 * i, 8);
        }
        sh.stop = 0;
        bar_init_done();
    }
    if (warp == 8) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The block holds all of TMEM, so its first column is 0: a constant, which
    // keeps the products' addresses in uniform registers.
    constexpr uint32_t tmem = 0;
    constexpr uint32_t t_dq = tmem + 384;
    constexpr bool kAhead = DP == 64;
    // Columns of a tile's S and dP and of the next tile's S; moved on from tile to tile.
    struct Place {
        uint32_t s = tmem, dp = tmem + 128, next = tmem + 256;
        __device__ __forceinline__ void move()
        {
            const uint32_t t = next;
            next = kAhead ? dp : s;
            if (kAhead) dp = s;
            s = t;
        }
    };
    auto turn = [](uint32_t bar, int j) { return bar + 8 * (j & 1); };
    auto phase = [](int j) { return static_cast<uint32_t>(j >> 1) & 1u; };
    volatile int* stop = &sh.stop;

    if (warp == 9) {
        regs_down<h3qk_core::kOtherRegs>();
        int issued = 0;
        if (lane == 0 && n > 0) {
            bar_expect(own, 2 * Shape::kTileBytes);
            load_tile(q_smem, &map_q, Shape::kBlocks, s.row0 + tile_row, head, s.item, own);
            load_tile(do_smem, &map_do, Shape::kBlocks, s.row0 + tile_row, head, s.item, own);
            for (int i = 0; i < 2 * n; ++i) {
                const int st = i % kStages;
                if (!bar_wait(empty + 8 * st, ((i / kStages) & 1) ^ 1, stop)) break;
                bar_expect(full + 8 * st, Shape::kTileBytes);
                load_tile(ring + st * Shape::kTileBytes, (i & 1) ? &map_v : &map_k, Shape::kBlocks,
                          s.k0 + (i >> 1) * kTile, kv_head, s.item, full + 8 * st);
                issued = i + 1;
            }
        }
        __syncwarp();
        if (fix) {
            // Keys of the last tile that no row of the block sees: cleared,
            // for dq multiplies ds = 0 with them.  (dp of such keys is not used.)
            const int i = 2 * n - 2, st = i % kStages;
            if (bar_wait(full + 8 * st, (i / kStages) & 1, stop)) {
                clear_rows(ring + st * Shape::kTileBytes, Shape::kBlocks, seen - (n - 1) * kTile);
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(fixed);
            }
        }
        __syncwarp();
        if (*stop && lane == 0) {
            if (n > 0)
                for (int t = 0; t < kMaxTries && !bar_test(own, 0); ++t) {}
            drain_loads(full, kStages, issued);
        }
    } else if (warp == 8) {
        regs_down<h3qk_core::kOtherRegs>();
        if (n > 0) {
            constexpr uint32_t shape_s = mma_shape(BF16, 128, kTile, false);
            constexpr uint32_t shape_d = mma_shape(BF16, 128, DP, true);
            const int steps = (p.dim + 15) / 16;
            auto tile_at = [&](int i) { return ring + (i % kStages) * Shape::kTileBytes; };
            auto loaded = [&](int i) { return bar_wait(full + 8 * (i % kStages), (i / kStages) & 1, stop); };
            auto free = [&](int i) { return empty + 8 * (i % kStages); };
            auto scores = [&](int j, uint32_t to) {
                if (!loaded(2 * j)) return false;
                if (fix && j == n - 1 && !bar_wait(fixed, 0, stop)) return false;
                product_rows<DP>(to, q_smem, tile_at(2 * j), steps, shape_s, turn(s_full, j));
                return true;
            };
            auto dprobs = [&](int j, uint32_t to) {
                if (!loaded(2 * j + 1)) return false;
                product_rows<DP>(to, do_smem, tile_at(2 * j + 1), steps, shape_s, turn(dp_full, j));
                signal(free(2 * j + 1));
                return true;
            };
            Place at;
            bool ok = bar_wait(own, 0, stop) && scores(0, at.s) && dprobs(0, at.dp) && (n < 2 || scores(1, at.next));
            for (int j = 0; j < n && ok; ++j, at.move()) {
                if (kAhead && j + 1 < n) {
                    ok = bar_wait(turn(s_free, j), phase(j), stop);
                    tc_fence_after();
                    ok = ok && dprobs(j + 1, at.s);
                }
                ok = ok && bar_wait(turn(ds_ready, j), phase(j), stop);
                if (!ok) break;
                tc_fence_after();
                product_sum(t_dq, at.dp, tile_at(2 * j), shape_d, j > 0, free(2 * j));
                if (!kAhead && j + 1 < n) ok = dprobs(j + 1, at.dp);
                if (ok && j + 2 < n) ok = scores(j + 2, kAhead ? at.dp : at.s);
            }
            if (ok) signal(done);
            __syncwarp();
            if (*stop && elect_lane()) drain_products(smem_addr(&sh.drain));
        }
        __syncwarp();
    } else if (warp < 8) {
        regs_up<h3qk_core::kMathRegs>();
        const int g = warp >> 2, r = threadIdx.x & 127;
        const int i_row = tile_row + r;
        const bool has = i_row < s.rows;
        const int64_t row = s.row0 + i_row;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        // delta = dout . out of the row; each half of the warps takes every other
        // 8 channels.  (out is rounded to its type, which is most of dq's error
        // on rows with a few heavy keys; the exact delta is known only after the
        // loop, in time for dk.)
        float part = 0.0f, off = 0.0f;
        if (has) {
            const uint16_t* o = p.out + s.item * p.os.item + head * p.os.head + row * p.os.row;
            const uint16_t* d = p.dout + s.item * p.dos.item + head * p.dos.head + row * p.dos.row;
            for (int c = 8 * g; c < p.dim; c += 16) {
                const uint4 ov = __ldg(reinterpret_cast<const uint4*>(o + c));
                const uint4 dv = __ldg(reinterpret_cast<const uint4*>(d + c));
                const uint32_t ow[4] = {ov.x, ov.y, ov.z, ov.w}, dw[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 a = widen_pair<BF16>(ow[e]), b = widen_pair<BF16>(dw[e]);
                    part = fmaf(a.x, b.x, part);
                    part = fmaf(a.y, b.y, part);
                    off = fmaf(fmaf(fabsf(a.x), kRound<BF16>, kTiny<BF16>), fabsf(b.x), off);
                    off = fmaf(fmaf(fabsf(a.y), kRound<BF16>, kTiny<BF16>), fabsf(b.y), off);
                }
            }
        }
        sh.delta[g][r] = part;
        sh.lse[g][r] = off;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float delta = sh.delta[0][r] + sh.delta[1][r];
        const float most = 2.0f * (sh.lse[0][r] + sh.lse[1][r]);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (g == 0) reinterpret_cast<float2*>(sh.lse)[r] = make_float2(delta - most, delta + most);
        const int64_t stat = (static_cast<int64_t>(s.item) * p.heads + head) * p.q_rows + row;
        float lse = INFINITY;  // p = 0
        if (has) {
            const float v = __ldg(p.lse + stat);
            if (v != -INFINITY) lse = v * h3qk_core::kLog2e;
        }
        const int lim = h3qk_core::limit_of(s, p.causal, i_row);
        const int lim_first = h3qk_core::limit_of(s, p.causal, tile_row);
        const Bend bend = h3qk_core::bend_of(p, head);
        const float c = p.scale * h3qk_core::kLog2e;
        const uint64_t cc = pair(c, c), nl = pair(-lse, -lse), nd = pair(-delta, -delta);
        uint64_t exact[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) exact[e] = pair(0.0f, 0.0f);
        bool ok = true;
        Place at;
        for (int j = 0; j < n; ++j, at.move()) {
            ok = bar_wait(turn(s_full, j), phase(j), stop);
            if (!ok) break;
            tc_fence_after();
            uint32_t sr[2][32];
            tmem_ld32(sr[0], at.s + lanes + 64 * g);
            tmem_ld32(sr[1], at.s + lanes + 64 * g + 32);
            tmem_wait_ld(sr[0]);
            tmem_wait_ld(sr[1]);
            if constexpr (kAhead) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(turn(s_free, j));
            }
            const float far = static_cast<float>(s.start + i_row - j * kTile - 64 * g);
            const bool edge = (j + 1) * kTile > lim_first;
            const int left = lim - j * kTile - 64 * g;
            uint64_t pp[2][16];                            // p
            uint64_t kp[BENDS & h3qk_core::kCapped ? 2 : 1][16];  // and with a cap 1 - tanh^2
            // Tiles that some row sees only in part have their own code: the
            // comparisons would cost every tile a third of its time.
            auto probabilities = [&](auto at_edge) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        uint64_t z[2];
                    [[maybe_unused]] uint64_t keep[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            z[i] = pair(__uint_as_float(sr[b][2 * (e + i)]), __uint_as_float(sr[b][2 * (e + i) + 1]));
                        if constexpr (BENDS != h3qk_core::kPlain)
                            h3qk_core::bend_four<BENDS, true>(z, bend, far - static_cast<float>(32 * b + 2 * e), -1.0f, keep);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float lo, hi;
                            unpair(lo, hi, BENDS == h3qk_core::kPlain ? fma_pair(z[i], cc, nl) : add_pair(z[i], nl));
                            lo = exp2_fast(lo);
                            hi = exp2_fast(hi);
                            if constexpr (decltype(at_edge)::value) {
                                if (32 * b + 2 * (e + i) >= left) lo = 0.0f;
                                if (32 * b + 2 * (e + i) + 1 >= left) hi = 0.0f;
                            }
                            pp[b][e + i] = pair(lo, hi);
                            if constexpr (BENDS & h3qk_core::kCapped) kp[b][e + i] = keep[i];
                        }
                    }
            };
            if (edge) probabilities(std::true_type{});
            else probabilities(std::false_type{});
            ok = bar_wait(turn(dp_full, j), phase(j), stop);
            if (!ok) break;
            tc_fence_after();
            auto gradients = [&](auto at_edge) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t dp[32], w[16];
                    tmem_ld32(dp, at.dp + lanes + 64 * g + 32 * b);
                    tmem_wait_ld(dp);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float lo = __uint_as_float(dp[2 * e]), hi = __uint_as_float(dp[2 * e + 1]);
                        if constexpr (decltype(at_edge)::value) {  // values that the row does not see may be anything
                            if (32 * b + 2 * e >= left) lo = 0.0f;
                            if (32 * b + 2 * e + 1 >= left) hi = 0.0f;
                        }
                        const uint64_t t = pair(lo, hi);
                        exact[e & 3] = fma_pair(pp[b][e], t, exact[e & 3]);
                        uint64_t d = mul_pair(pp[b][e], add_pair(t, nd));
                        if constexpr (BENDS & h3qk_core::kCapped) d = mul_pair(d, kp[b][e]);
                        unpair(lo, hi, d);
                        w[e] = round_pair<BF16>(lo, hi);
                    }
                    tmem_st16(at.dp + lanes + 64 * g + 16 * b, w);
                }
            };
            if (edge) gradients(std::true_type{});
            else gradients(std::false_type{});
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(turn(ds_ready, j));
        }
        if (ok && n > 0) ok = bar_wait(done, 0, stop);
        tc_fence_after();
        // For dk, delta = sum_j p dp without the rounding of out.  That needs all
        // the keys that out and lse stem from; where other calls took some of
        // them, the sum differs from dout . out by more than out's rounding (and as
        // much again for that of p) explains, and is held to that.
        float lo, hi;
        unpair(lo, hi, add_pair(add_pair(exact[0], exact[1]), add_pair(exact[2], exact[3])));
        asm volatile("bar.sync 1, 256;" ::: "memory");  // all have read the first delta
        sh.delta[g][r] = ok ? lo + hi : given_up();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (g == 0 && has) {
            const float2 within = reinterpret_cast<const float2*>(sh.lse)[r];
            const float sum = sh.delta[0][r] + sh.delta[1][r];
            p.delta[stat] = sum == sum ? fminf(fmaxf(sum, within.x), within.y) : sum;
        }
        uint16_t* dst = p.dq + s.item * p.dqs.item + head * p.dqs.head + row * p.dqs.row;
        write_row<BF16, DP / 2>(dst, t_dq + lanes + g * (DP / 2), g * (DP / 2), p.dim, ok ? p.scale : given_up(),
                                !(has && n > 0), i_row < s.span);
        tc_fence_before();
    } else {
        regs_down<h3qk_core::kOtherRegs>();
    }
    __syncthreads();
    if (threadIdx.x == 0 && *stop) atomicAdd(p.stuck, 1u);
    if (warp == 8) {
        tc_fence_after();
        tmem_free(sh.tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// dk, dv: a block's 128 keys of a K/V head against the query tiles that see
// them, of every head that shares it.
//   tensor unit   S0 dP0 | dV0 S1 dK0 dP1 | dV1 S2 dK1 dP2 | ...
// (S = k q^T and dP = v dout^T: the keys are the lanes.)  p of the next tile
// is computed while dK and dP run, ds while dV and S run.
// ---------------------------------------------------------------------------
template <bool BF16, int DP, int BENDS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                         const __grid_constant__ Params p)
{
    using Shape = BwdShape<DP>;
    constexpr int kStages = Shape::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    BwdShared& sh = *reinterpret_cast<BwdShared*>(smem_raw + Shape::kTiles);
    const uint32_t base = smem_addr(smem_raw);
    if (base & 1023u) {  // the swizzle needs it; the launch gives it
        if (threadIdx.x == 0) atomicAdd(p.stuck, 1u);
        return;
    }
    const uint32_t k_smem = base, v_smem = base + Shape::kTileBytes, ring = base + 2 * Shape::kTileBytes;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const Place3 block = place_of(p.causal, false, p.kv_heads, p.batch);
    const int kv_head = block.head;

    Stretch s;
    if (!h3qk_core::find_stretch(s, p, block.tile, block.item, kTile, true)) return;
    const int tile_key = s.tile * kTile;
    const int q_tiles = (s.rows + kTile - 1) / kTile;
    // First query tile that sees any of the keys; none if the keys do not exist.
    const int first_row = !p.causal || tile_key < s.prefix ? 0 : max(tile_key - s.start, 0);
    const int q_first = tile_key < s.keys ? min(first_row / kTile, q_tiles) : q_tiles;
    const int per_head = q_tiles - q_first;
    const int n = per_head * p.group;
    // Rows of each head's last query tile past the rows that attend.
    const bool fix = s.rows % kTile != 0 && s.row0 + s.rows < p.q_rows;

    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty), own = smem_addr(&sh.own);
    const uint32_t s_full = smem_addr(sh.s_full), dp_full = smem_addr(sh.dp_full);
    const uint32_t p_ready = smem_addr(sh.p_ready), ds_ready = smem_addr(sh.ds_ready);
    const uint32_t st_full = smem_addr(sh.st_full), st_empty = smem_addr(sh.st_empty);
    const uint32_t fixed = smem_addr(sh.fixed), done = smem_addr(&sh.done);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, 1);
            bar_init(empty + 8 * i, 1);
        }
        bar_init(own, 1);
        for (int i = 0; i < 2; ++i) bar_init(fixed + 8 * i, 1);
        bar_init(done, 1);
        bar_init(smem_addr(&sh.drain), 1);
        bar_init(s_full, 1);
        bar_init(s_full + 8, 1);
        bar_init(dp_full, 1);
        bar_init(p_ready, 8);
        bar_init(p_ready + 8, 8);
        bar_init(ds_ready, 8);
        for (int i = 0; i < 2; ++i) {
            bar_init(st_full + 8 * i, 1);
            bar_init(st_empty + 8 * i, 8);
        }
        sh.stop = 0;
        bar_init_done();
    }
    if (warp == 8) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The block holds all of TMEM, so its first column is 0: a constant, which
    // keeps the products' addresses in uniform registers.
    constexpr uint32_t tmem = 0;
    // S is double-buffered where TMEM has the room (up to 64 channels): the next
    // tile's S is then done before its turn.
    constexpr int kScores = DP == 64 ? 2 : 1;
    const uint32_t t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 256 + DP;
    auto t_s = [&](int i) { return kScores == 2 && (i & 1) ? tmem + 384 : tmem; };
    auto s_bar = [&](int i) { return s_full + 8 * (kScores == 2 ? i & 1 : 0); };
    auto s_phase = [&](int i) { return static_cast<uint32_t>(kScores == 2 ? i >> 1 : i) & 1u; };
    volatile int* stop = &sh.stop;
    auto head_of = [&](int i) { return kv_head * p.group + i / per_head; };
    auto row_of = [&](int i) { return (q_first + i % per_head) * kTile; };

    if (warp == 9) {
        regs_down<h3qk_core::kOtherRegs>();
        int issued = 0;
        if (lane == 0 && n > 0) {
            bar_expect(own, 2 * Shape::kTileBytes);
            load_tile(k_smem, &map_k, Shape::kBlocks, s.k0 + tile_key, kv_head, s.item, own);
            load_tile(v_smem, &map_v, Shape::kBlocks, s.k0 + tile_key, kv_head, s.item, own);
            for (int i = 0; i < 2 * n; ++i) {
                const int st = i % kStages;
                if (!bar_wait(empty + 8 * st, ((i / kStages) & 1) ^ 1, stop)) break;
                bar_expect(full + 8 * st, Shape::kTileBytes);
                load_tile(ring + st * Shape::kTileBytes, (i & 1) ? &map_do : &map_q, Shape::kBlocks,
                          s.row0 + row_of(i >> 1), head_of(i >> 1), s.item, full + 8 * st);
                issued = i + 1;
            }
        }
        __syncwarp();
        if (*stop && lane == 0) {
            if (n > 0)
                for (int t = 0; t < kMaxTries && !bar_test(own, 0); ++t) {}
            drain_loads(full, kStages, issued);
        }
    } else if (warp == 10) {
        regs_down<h3qk_core::kOtherRegs>();
        // Statistics of each query tile: -lse in powers of two (-infinite where
        // the row sees nothing or does not attend, so that p = 0), and -delta.
        // A tile's loads are all in flight before the turn of the tile before it.
        float l[4], d[4];
        auto fetch = [&](int i) {
            const float* lse = p.lse + (static_cast<int64_t>(s.item) * p.heads + head_of(i)) * p.q_rows + s.row0;
            const float* delta = p.delta + (lse - p.lse);
            const int r0 = row_of(i) + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = min(r0 + 32 * e, s.rows - 1);
                l[e] = __ldg(lse + r);
                d[e] = __ldcg(delta + r);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = r0 + 32 * e < s.rows;
                l[e] = there && l[e] != -INFINITY ? fmaf(l[e], -h3qk_core::kLog2e, kLift<BF16>) : -INFINITY;
                d[e] = there ? d[e] * -kDrop<BF16> : 0.0f;
            }
        };
        if (n > 0) fetch(0);
        for (int i = 0; i < n; ++i) {
            if (!bar_wait(st_empty + 8 * (i & 1), ((i >> 1) & 1) ^ 1, stop)) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sh.lse[i & 1][32 * e + lane] = l[e];
                sh.delta[i & 1][32 * e + lane] = d[e];
            }
            __syncwarp();
            if (lane == 0) bar_arrive(st_full + 8 * (i & 1));
            if (i + 1 < n) fetch(i + 1);
            if (fix && i % per_head == per_head - 1) {
                // The head's last tile: rows that do not attend are cleared, for
                // dv and dk multiply p = ds = 0 with them.  The wait above says
                // that tile i - 2 is done, so this tile's stages are in their
                // present use; the products wait for `fixed` before the next.
                bool ok = true;
                for (int k = 2 * i; k < 2 * i + 2 && ok; ++k) {
                    ok = bar_wait(full + 8 * (k % kStages), (k / kStages) & 1, stop);
                    if (ok) clear_rows(ring + (k % kStages) * Shape::kTileBytes, Shape::kBlocks, s.rows % kTile);
                }
                if (!ok) break;
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(fixed + 8 * (i / per_head & 1));
            }
        }
    } else if (warp == 8) {
        regs_down<h3qk_core::kOtherRegs>();
        if (n > 0) {
            constexpr uint32_t shape_s = mma_shape(BF16, 128, kTile, false);
            constexpr uint32_t shape_d = mma_shape(BF16, 128, DP, true);
            const int steps = (p.dim + 15) / 16;
            auto tile_at = [&](int i) { return ring + (i % kStages) * Shape::kTileBytes; };
            auto loaded = [&](int i) { return bar_wait(full + 8 * (i % kStages), (i / kStages) & 1, stop); };
            auto free = [&](int i) { return empty + 8 * (i % kStages); };
            // The clearing warp is never a head ahead of the next but one to be waited
            // for: two barriers tell its turns apart.
            auto cleared = [&](int h) { return bar_wait(fixed + 8 * (h & 1), (h >> 1) & 1, stop); };
            auto scores = [&](int i) {
                if (!loaded(2 * i)) return false;
                if (fix && i % per_head == per_head - 1 && !cleared(i / per_head)) return false;
                product_rows<DP>(t_s(i), k_smem, tile_at(2 * i), steps, shape_s, s_bar(i));
                return true;
            };
            auto dprobs = [&](int i) {
                if (!loaded(2 * i + 1)) return false;
                product_rows<DP>(t_dp, v_smem, tile_at(2 * i + 1), steps, shape_s, dp_full);
                return true;
            };
            bool ok = bar_wait(own, 0, stop) && scores(0) && dprobs(0) && (kScores == 1 || n < 2 || scores(1));
            for (int i = 0; i < n && ok; ++i) {
                ok = bar_wait(p_ready + 8 * (i & 1), (i >> 1) & 1, stop);
                if (!ok) break;
                tc_fence_after();
                product_sum(t_dv, t_s(i), tile_at(2 * i + 1), shape_d, i > 0, free(2 * i + 1));
                if (i + kScores < n) ok = scores(i + kScores);
                ok = ok && bar_wait(ds_ready, i & 1, stop);
                if (!ok) break;
                tc_fence_after();
                product_sum(t_dk, t_dp, tile_at(2 * i), shape_d, i > 0, free(2 * i));
                if (i + 1 < n) ok = dprobs(i + 1);
            }
            if (ok) signal(done);
            __syncwarp();
            if (*stop && elect_lane()) drain_products(smem_addr(&sh.drain));
        }
        __syncwarp();
    } else if (warp < 8) {
        regs_up<h3qk_core::kMathRegs>();
        const int g = warp >> 2, r = threadIdx.x & 127;
        const int key = tile_key + r;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        // Row i sees the key when i >= from.
        const int from = p.causal && key >= s.prefix ? key - s.start : -h3qk_core::kFar;
        const int last_key = min(tile_key + kTile, s.keys) - 1;
        const int from_last = p.causal && last_key >= s.prefix ? last_key - s.start : -h3qk_core::kFar;
        const float c = p.scale * h3qk_core::kLog2e;
        const uint64_t cc = pair(c, c), drop = pair(kDrop<BF16>, kDrop<BF16>);
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int row0 = row_of(i) + 64 * g;
            const Bend bend = h3qk_core::bend_of(p, head_of(i));
            ok = bar_wait(st_full + 8 * (i & 1), (i >> 1) & 1, stop) && bar_wait(s_bar(i), s_phase(i), stop);
            if (!ok) break;
            tc_fence_after();
            const ulonglong2* nl = reinterpret_cast<const ulonglong2*>(sh.lse[i & 1] + 64 * g);
            const ulonglong2* nd = reinterpret_cast<const ulonglong2*>(sh.delta[i & 1] + 64 * g);
            uint32_t sr[2][32];
            tmem_ld32(sr[0], t_s(i) + lanes + 64 * g);
            tmem_ld32(sr[1], t_s(i) + lanes + 64 * g + 32);
            tmem_wait_ld(sr[0]);
            tmem_wait_ld(sr[1]);
            const bool edge = row_of(i) < from_last;
            const int hidden = from - row0;  // queries of this half that do not see the key
            const float far = static_cast<float>(s.start + row0 - key);
            uint64_t pp[2][16];
            auto probabilities = [&](auto at_edge) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const ulonglong2 l2 = nl[(16 * b + e) >> 1];
                        uint64_t z[2];
                    [[maybe_unused]] uint64_t keep[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            z[i] = pair(__uint_as_float(sr[b][2 * (e + i)]), __uint_as_float(sr[b][2 * (e + i) + 1]));
                        if constexpr (BENDS != h3qk_core::kPlain)
                            h3qk_core::bend_four<BENDS, true>(z, bend, far + static_cast<float>(32 * b + 2 * e), 1.0f, keep);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint64_t l = i ? l2.y : l2.x;
                            float lo, hi;
                            unpair(lo, hi, BENDS == h3qk_core::kPlain ? fma_pair(z[i], cc, l) : add_pair(z[i], l));
                            lo = exp2_fast(lo);
                            hi = exp2_fast(hi);
                            if constexpr (decltype(at_edge)::value) {
                                if (32 * b + 2 * (e + i) < hidden) lo = 0.0f;
                                if (32 * b + 2 * (e + i) + 1 < hidden) hi = 0.0f;
                            }
                            pp[b][e + i] = pair(lo, hi);
                            w[e + i] = round_pair<BF16>(lo, hi);
                            if constexpr (BENDS & h3qk_core::kCapped) pp[b][e + i] = mul_pair(pp[b][e + i], keep[i]);
                        }
                    }
                    tmem_st16(t_s(i) + lanes + 64 * g + 16 * b, w);
                }
            };
            if (edge) probabilities(std::true_type{});
            else probabilities(std::false_type{});
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready + 8 * (i & 1));
            ok = bar_wait(dp_full, i & 1, stop);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t dp[32], w[16];
                tmem_ld32(dp, t_dp + lanes + 64 * g + 32 * b);
                tmem_wait_ld(dp);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const ulonglong2 d2 = nd[(16 * b + e) >> 1];
                    const uint64_t d = (e & 1) ? d2.y : d2.x;
                    uint64_t t = pair(__uint_as_float(dp[2 * e]), __uint_as_float(dp[2 * e + 1]));
                    if constexpr (BF16) t = add_pair(t, d);
                    else t = fma_pair(t, drop, d);
                    float lo, hi;
                    unpair(lo, hi, mul_pair(pp[b][e], t));
                    w[e] = round_pair<BF16>(lo, hi);
                }
                tmem_st16(t_dp + lanes + 64 * g + 16 * b, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(ds_ready);
                bar_arrive(st_empty + 8 * (i & 1));
            }
        }
        if (ok && n > 0) ok = bar_wait(done, 0, stop);
        tc_fence_after();
        const int64_t row = s.k0 + key;
        // keys that some row sees; others get zeros, whatever they hold
        const bool zero = !(n > 0 && key < s.keys && from < s.rows);
        if (g == 0)
            write_row<BF16, DP>(p.dv + s.item * p.dvs.item + kv_head * p.dvs.head + row * p.dvs.row, t_dv + lanes, 0,
                                p.dim, ok ? kDrop<BF16> : given_up(), zero, key < s.span);
        else
            write_row<BF16, DP>(p.dk + s.item * p.dks.item + kv_head * p.dks.head + row * p.dks.row, t_dk + lanes, 0,
                                p.dim, ok ? p.scale : given_up(), zero, key < s.span);
        tc_fence_before();
    } else {
        regs_down<h3qk_core::kOtherRegs>();
    }
    __syncthreads();
    if (threadIdx.x == 0 && *stop) atomicAdd(p.stuck, 1u);
    if (warp == 8) {
        tc_fence_after();
        tmem_free(sh.tmem, 512);
    }
}

template <bool BF16, int DP, int BENDS>
cudaError_t launch(const Params& p, const h3qk_core::Maps& m, cudaStream_t st)
{
    constexpr int smem = BwdShape<DP>::kTiles + static_cast<int>(sizeof(BwdShared));
    static_assert(smem <= 227 * 1024, "tiles and barriers exceed a block's shared memory");
    static bool done[2][64] = {};
    auto* dq = attention_dq_kernel<BF16, DP, BENDS>;
    auto* dkv = attention_dkv_kernel<BF16, DP, BENDS>;
    cudaError_t e = h3qk_core::ready(dq, smem, done[0]);
    if (e == cudaSuccess) e = h3qk_core::ready(dkv, smem, done[1]);
    if (e != cudaSuccess) return e;
    if (p.q_rows > 0) {
        const dim3 grid(static_cast<unsigned>(h3qk_core::tiles_of(p, p.q_rows, kTile)), p.heads, p.batch);
        dq<<<grid, kThreads, smem, st>>>(m.q, m.k, m.v, m.dout, p);
        h3qk_internal_count_launch();
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (p.kv_rows > 0) {
        const dim3 grid(static_cast<unsigned>(h3qk_core::tiles_of(p, p.kv_rows, kTile)), p.kv_heads, p.batch);
        dkv<<<grid, kThreads, smem, st>>>(m.q, m.k, m.v, m.dout, p);
        h3qk_internal_count_launch();
        e = cudaGetLastError();
    }
    return e;
}

template <bool BF16, int DP>
cudaError_t by_bends(const Params& p, const h3qk_core::Maps& m, cudaStream_t st)
{
    using namespace h3qk_core;
    if (p.cap > kWideCap) return launch<BF16, DP, kCapped | kSloped | kWide>(p, m, st);  // (slopes of 0 where there are none)
    if (p.cap > 0.0f) return p.slopes ? launch<BF16, DP, kCapped | kSloped>(p, m, st) : launch<BF16, DP, kCapped>(p, m, st);
    return p.slopes ? launch<BF16, DP, kSloped>(p, m, st) : launch<BF16, DP, kPlain>(p, m, st);
}

template <bool BF16>
cudaError_t by_shape(const Params& p, const h3qk_core::Maps& m, cudaStream_t st)
{
    return p.dim <= 64 ? by_bends<BF16, 64>(p, m, st) : by_bends<BF16, 128>(p, m, st);
}

}  // namespace

cudaError_t h3qk_core::backward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st)
{
    return bf16 ? by_shape<true>(p, m, st) : by_shape<false>(p, m, st);
}
