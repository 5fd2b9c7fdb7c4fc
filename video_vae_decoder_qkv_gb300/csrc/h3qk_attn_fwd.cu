// Attention forward, many rows: one block takes 256 query rows of a head and
// streams its keys and values once.
//
//   s = bend(q k^T),  m = running row maximum,  p = 2^(s - m),
//   o = sum p v / sum p,  lse = ln(sum e^s)
//
// Two groups of four warps own 128 rows each, one thread a row, so the
// softmax needs no exchange between threads.  One thread issues the matrix
// products, one warp the tile loads.  The products of one group run while
// the other group computes its softmax:
//   tensor unit   S0 S1 | O0 S0' O1 S1' | ...      (S = q k^T, O += p v)
// P replaces S in TMEM (as 16-bit pairs) and is the product's A operand from
// there; the tensor unit works in order, so a new S may be issued behind the O
// that reads P from the same columns.  TMEM's 512 columns hold both O and two
// S at head_dim 128; up to 64 they hold three S, which the groups' tiles take
// in turn, so that a group finds its next S done when it has left its last P.  O stays in TMEM; it is rescaled only
// when some row's maximum has grown by more than 2^8, otherwise the old
// maximum serves on (p then reaches 2^8, far from any overflow; for fp16 all
// p are kept 2^7 larger, so that flat rows do not fall into subnormals).
//
// P is rounded to the input type: that is what the tensor unit multiplies.
// The row sum adds the unrounded p in binary32, O accumulates in binary32.
//
// Bound: at head_dim 128 by the tensor unit (2 x 512 cycles a tile and group;
// a group's softmax takes about 1,100 and overlaps the other group's products).
// 40 heads of 8160 x 8160 x 128, bf16: 0.79 ms in short runs, 1.73 PFLOP/s, 93 %
// of the rate that short products measured; 0.86 ms where passes follow one
// another under the power cap, 93 % of the rate of products that do.
// Up to 64 the softmax takes longer than the products (per score one 2^x at 32 a
// cycle and SM, and about four instructions), but neither is busy all the time:
// counters show the tensor unit and 2^x at 48 % each, for a warp's turn is a chain
// of waits (TMEM read, maximum, 2^x, TMEM write, arrival) with one other warp to
// fill it.  32 heads of 8192 x 8192 x 64, fp16: 0.47 ms, 1.17 PFLOP/s.  With a
// cap, two 2^x and a quarter of a reciprocal a score and the same chain: 0.91
// PFLOP/s at 128, 0.53 at 64.
// The issuing warp runs its loop converged: with one lane inside a divergent
// branch the products' operands left the uniform registers and issuing them
// took longer than computing them (1.01 instead of 1.64 PFLOP/s).
#include "h3qk_attn.cuh"

#include <type_traits>

namespace {

using namespace h3qk_tc;
using h3qk_core::Bend;
using h3qk_core::Params;
using h3qk_core::Stretch;

constexpr int kTile = 128;             // rows of a group, keys of a tile
constexpr int kThreads = 384;          // 2 x 4 softmax warps; products, loads, two idle
constexpr float kSlack = 8.0f;         // log2: growth of the maximum that is tolerated
constexpr int kBlockBytes = 128 * 128; // 64 columns of a tile

template <int DP>
struct FwdShape {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kScores = DP == 128 ? 2 : 3;  // S buffers
    static constexpr uint32_t kOut = 128 * kScores;    // first column of O
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes;
};

struct FwdShared {
    uint64_t full[8], empty[8];
    uint64_t q_full, fixed;
    uint64_t s_full[4], p_ready[4], o_done[2], all_done[2], drain;
    uint32_t tmem;
    int stop;
};

// Where tile number t of a call lies.  A head's tiles follow one another, so
// that its keys stay in L2.  Causal rows see more keys the later they are:
// there the longest tiles of all heads go first, and the shortest fill the end.
struct Place {
    int tile, head, item;
};
__device__ __forceinline__ Place place_of(const Params& p, int t)
{
    Place at;
    if (p.causal) {
        at.head = t % p.heads;
        t /= p.heads;
        at.item = t % p.batch;
        at.tile = p.tiles - 1 - t / p.batch;
    } else {
        at.tile = t % p.tiles;
        t /= p.tiles;
        at.head = t % p.heads;
        at.item = t / p.heads;
    }
    return at;
}

template <bool BF16, int DP, int BENDS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p)
{
    using Shape = FwdShape<DP>;
    constexpr int kStages = Shape::kStages;
    constexpr float kShift = BF16 ? 0.0f : 7.0f;
    extern __shared__ uint8_t smem_raw[];
    __shared__ FwdShared sh;
    h3qk_ops::allow_dependents();
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = base, ring = base + 2 * Shape::kTileBytes;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool cut = blockIdx.x >= p.whole;  // one of the parts of a tail tile
    const int part = cut ? (blockIdx.x - p.whole) % p.parts : 0;
    const Place at = place_of(p, cut ? p.whole + (blockIdx.x - p.whole) / p.parts : blockIdx.x);
    const int head = at.head, kv_head = head / p.group;

    Stretch s;
    if (!h3qk_core::find_stretch(s, p, at.tile, at.item, 2 * kTile, false)) return;
    const int tile_row = s.tile * 2 * kTile;
    int n[2], seen = 0;  // tiles of each group, keys that any row of the block sees
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = tile_row + g * kTile;
        const int last = min(first + kTile, s.rows) - 1;
        const int lim = last < first ? 0 : max(h3qk_core::limit_of(s, p.causal, last), 0);
        n[g] = (lim + kTile - 1) / kTile;
        seen = max(seen, lim);
    }
    int n_all = max(n[0], n[1]), j0 = 0;  // tiles of this block; the first of them
    if (cut) {
        const int each = (n_all + p.parts - 1) / p.parts, last = n_all;
        j0 = min(part * each, last);
        n_all = min(last - j0, each);
#pragma unroll
        for (int g = 0; g < 2; ++g) n[g] = min(max(n[g] - j0, 0), n_all);
    }
    const int key0 = j0 * kTile;
    // Rows of the last tile that no row of the block sees: unwritten cache
    // rows, another document's, later tokens.  They are cleared (0 * NaN is
    // NaN, even with p = 0); past the tensor's end the loads give zeros.
    const bool fix = n_all > 0 && key0 + n_all * kTile > seen && s.k0 + seen < p.kv_rows;

    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t s_full = smem_addr(sh.s_full), p_ready = smem_addr(sh.p_ready), o_done = smem_addr(sh.o_done);
    const uint32_t all_done = smem_addr(sh.all_done);  // the last O, which is waited for by its own barrier
    const uint32_t q_full = smem_addr(&sh.q_full), fixed = smem_addr(&sh.fixed);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, 1);
            bar_init(empty + 8 * i, 1);
        }
        for (int g = 0; g < 2; ++g) {
            // Two of these for each group, taken in turn by its tiles: with S done
            // ahead, one side may come to a phase before the other has left the last.
            for (int i = 0; i < 2; ++i) {
                bar_init(s_full + 8 * (2 * g + i), 1);
                bar_init(p_ready + 8 * (2 * g + i), 4);
            }
            bar_init(o_done + 8 * g, 1);
            bar_init(all_done + 8 * g, 1);
        }
        bar_init(q_full, 1);
        bar_init(fixed, 1);
        bar_init(smem_addr(&sh.drain), 1);
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
    volatile int* stop = &sh.stop;
    auto turn = [](uint32_t bar, int g, int j) { return bar + 8 * (2 * g + (j & 1)); };
    auto phase = [](int j) { return static_cast<uint32_t>(j >> 1) & 1u; };

    if (warp > 9) {
        regs_down<h3qk_core::kOtherRegs>();
    } else if (warp == 9) {
        regs_down<h3qk_core::kOtherRegs>();
        // ---- tile loads: Q, then K and V tiles in turn ----------------------
        int issued = 0;
        bool ok = true;
        if (lane == 0 && n_all > 0) {
            tma_prefetch(&map_k);
            tma_prefetch(&map_v);
            bar_expect(q_full, 2 * Shape::kTileBytes);
            for (int g = 0; g < 2; ++g)
                for (int b = 0; b < Shape::kBlocks; ++b)
                    tma_load(q_smem + g * Shape::kTileBytes + b * kBlockBytes, &map_q, 64 * b,
                             s.row0 + tile_row + g * kTile, head, s.item, q_full);
            for (int i = 0; i < 2 * n_all && ok; ++i) {
                const int st = i % kStages;
                ok = bar_wait(empty + 8 * st, ((i / kStages) & 1) ^ 1, stop);
                if (!ok) break;
                bar_expect(full + 8 * st, Shape::kTileBytes);
                const int row = s.k0 + key0 + (i >> 1) * kTile;
                for (int b = 0; b < Shape::kBlocks; ++b)
                    tma_load(ring + st * Shape::kTileBytes + b * kBlockBytes, (i & 1) ? &map_v : &map_k, 64 * b, row,
                             kv_head, s.item, full + 8 * st);
                issued = i + 1;
            }
        }
        __syncwarp();
        if (fix) {
            const int i = 2 * n_all - 1, st = i % kStages;
            if (bar_wait(full + 8 * st, (i / kStages) & 1, stop)) {
                const int first = seen - key0 - (n_all - 1) * kTile;  // rows to keep
                for (int b = 0; b < Shape::kBlocks; ++b)
                    for (int o = first * 128 + lane * 16; o < kBlockBytes; o += 512)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + st * Shape::kTileBytes + b * kBlockBytes + o),
                                     "r"(0)
                                     : "memory");
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(fixed);
            }
        }
        __syncwarp();
        if (*stop && lane == 0) {
            // Given up: this block's loads must land before it leaves.
            if (n_all > 0)
                for (int t = 0; t < kMaxTries && !bar_test(q_full, 0); ++t) {}
            for (int i = max(0, issued - kStages); i < issued; ++i)
                for (int t = 0; t < kMaxTries && !bar_test(full + 8 * (i % kStages), (i / kStages) & 1); ++t) {}
        }
    } else if (warp == 8) {
        regs_down<h3qk_core::kOtherRegs>();
        // ---- matrix products ------------------------------------------------
        if (n_all > 0) {
            constexpr uint32_t shape_s = mma_shape(BF16, 128, kTile, false);
            constexpr uint32_t shape_o = mma_shape(BF16, 128, DP, true);
            const int steps = (p.dim + 15) / 16;
            auto release = [&](int i) {
                if (elect_lane()) mma_commit(empty + 8 * (i % kStages));
                __syncwarp();
            };
            auto loaded = [&](int i) { return bar_wait(full + 8 * (i % kStages), (i / kStages) & 1, stop); };
            auto tile_at = [&](int i) { return ring + (i % kStages) * Shape::kTileBytes; };
            // The groups take turns, and the turns take the S buffers in turn.  Each
            // tile is waited for in group 0's turn and released in group 1's, also
            // where one of them does not use it.
            uint32_t s_next = tmem, p_next = tmem;
            auto move = [&](uint32_t& at) { at = at + 128 == tmem + Shape::kOut ? tmem : at + 128; };
            auto scores = [&](auto group, int j) {
                constexpr int g = decltype(group)::value;
                if (j >= n_all) return true;
                if (g == 0 && !loaded(2 * j)) return false;
                if (j < n[g]) {
                    const uint64_t a = tile_desc(q_smem + g * Shape::kTileBytes, 16), b = tile_desc(tile_at(2 * j), 16);
                    if (elect_lane()) {
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k)
                            if (k < steps) {
                                constexpr int kStep = 32 >> 4, kNext = kBlockBytes >> 4;
                                const uint32_t off = (k >> 2) * kNext + (k & 3) * kStep;
                                mma_ss(s_next, a + off, b + off, shape_s, k > 0);
                            }
                        mma_commit(turn(s_full, g, j));
                    }
                    __syncwarp();
                }
                move(s_next);
                if (g == 1) release(2 * j);
                return true;
            };
            auto values = [&](auto group, int j) {
                constexpr int g = decltype(group)::value;
                if (g == 0 && !loaded(2 * j + 1)) return false;
                if (g == 0 && fix && j + 1 == n_all && !bar_wait(fixed, 0, stop)) return false;
                if (j < n[g]) {
                    if (!bar_wait(turn(p_ready, g, j), phase(j), stop)) return false;
                    tc_fence_after();
                    const uint64_t b = tile_desc(tile_at(2 * j + 1), kBlockBytes);
                    const uint32_t d = tmem + Shape::kOut + g * DP;
                    if (elect_lane()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            mma_ts(d, p_next + 8 * k, b + (k * 2048 >> 4), shape_o, j > 0 || k > 0);
                        mma_commit((j + 1 < n[g] ? o_done : all_done) + 8 * g);
                    }
                    __syncwarp();
                }
                move(p_next);
                if (g == 1) release(2 * j + 1);
                return true;
            };
            const std::integral_constant<int, 0> g0;
            const std::integral_constant<int, 1> g1;
            bool ok = bar_wait(q_full, 0, stop) && scores(g0, 0) && scores(g1, 0);
            if constexpr (Shape::kScores == 2) {
                for (int j = 0; j < n_all && ok; ++j)
                    ok = values(g0, j) && scores(g0, j + 1) && values(g1, j) && scores(g1, j + 1);
            } else {
                ok = ok && scores(g0, 1);
                for (int j = 0; j < n_all && ok; ++j)
                    ok = values(g0, j) && scores(g1, j + 1) && values(g1, j) && scores(g0, j + 2);
            }
            __syncwarp();
            if (*stop && elect_lane()) {
                const uint32_t drain = smem_addr(&sh.drain);
                mma_commit(drain);
                for (int t = 0; t < kMaxTries && !bar_test(drain, 0); ++t) {}
            }
        }
        __syncwarp();
    } else {
        regs_up<h3qk_core::kMathRegs>();
        // ---- softmax: one thread a row --------------------------------------
        const int g = warp >> 2;
        const int r = threadIdx.x & 127;
        const int i_row = tile_row + g * kTile + r;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_cols = tmem + Shape::kOut + g * DP + lanes;
        const int lim = h3qk_core::limit_of(s, p.causal, i_row);
        const int lim_first = h3qk_core::limit_of(s, p.causal, tile_row + g * kTile);
        const Bend bend = h3qk_core::bend_of(p, head);
        // Scores to powers of two: the bend gives exponents itself.
        const float c = BENDS != h3qk_core::kPlain ? 1.0f : p.scale * h3qk_core::kLog2e;
        const uint64_t cc = pair(c, c);
        float m = -INFINITY;
        uint64_t sum2 = pair(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < n[g] && ok; ++j) {
            ok = bar_wait(turn(s_full, g, j), phase(j), stop);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_cols = tmem + (2 * j + g) % Shape::kScores * 128 + lanes;
            uint32_t sr[4][32];
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_ld32(sr[b], s_cols + 32 * b);
#pragma unroll
            for (int b = 0; b < 4; ++b) tmem_wait_ld(sr[b]);
            const bool edge = key0 + (j + 1) * kTile > lim_first;  // some row sees the tile only in part
            const int left = lim - key0 - j * kTile;
            auto hide = [&](int b, int e, uint32_t as) {
                if (32 * b + e >= left) sr[b][e] = as;
            };
            auto bend_all = [&](auto at_edge) {
                const float far = static_cast<float>(s.start + i_row - key0 - j * kTile);
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        // Hidden scores may be NaN, and under a cap four share a reciprocal.
                        if constexpr (decltype(at_edge)::value)
#pragma unroll
                            for (int i = 0; i < 4; ++i) hide(b, e + i, 0u);
                        uint64_t z[2], keep[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            z[i] = pair(__uint_as_float(sr[b][e + 2 * i]), __uint_as_float(sr[b][e + 2 * i + 1]));
                        h3qk_core::bend_four<BENDS, false>(z, bend, far - static_cast<float>(32 * b + e), -1.0f, keep);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float lo, hi;
                            unpair(lo, hi, z[i]);
                            sr[b][e + 2 * i] = __float_as_uint(lo);
                            sr[b][e + 2 * i + 1] = __float_as_uint(hi);
                        }
                        if constexpr (decltype(at_edge)::value)
#pragma unroll
                            for (int i = 0; i < 4; ++i) hide(b, e + i, 0xff800000u);
                    }
            };
            if constexpr (BENDS & h3qk_core::kCapped) {
                if (edge) bend_all(std::true_type{});
                else bend_all(std::false_type{});
            } else {
                if constexpr (BENDS != h3qk_core::kPlain) bend_all(std::false_type{});
                if (edge) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 32; ++e) hide(b, e, 0xff800000u);
                }
            }
            float mx[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                mx[b] = fmaxf(__uint_as_float(sr[b][0]), __uint_as_float(sr[b][1]));
#pragma unroll
                for (int e = 2; e < 32; e += 2) mx[b] = max3(mx[b], __uint_as_float(sr[b][e]), __uint_as_float(sr[b][e + 1]));
            }
            const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
            if (__any_sync(0xffffffffu, (top - m) * c > kSlack)) {
                if (j > 0) {
                    const float f = top == -INFINITY ? 1.0f : exp2_fast((m - top) * c);
                    const uint64_t ff = pair(f, f);
                    sum2 = mul_pair(sum2, ff);
                    // (This S being done, all O but the last one are.)
                    ok = bar_wait(o_done + 8 * g, (j - 1) & 1, stop);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int d = 0; d < DP; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(o, o_cols + d);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(o_cols + d, o);
                    }
                }
                m = top;
            }
            const float mc = (m == -INFINITY ? 0.0f : m * c) - kShift;
            const uint64_t nm = pair(-mc, -mc);
            uint64_t part[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t pr[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float lo, hi;
                    unpair(lo, hi, fma_pair(pair(__uint_as_float(sr[b][2 * e]), __uint_as_float(sr[b][2 * e + 1])), cc, nm));
                    lo = exp2_fast(lo);
                    hi = exp2_fast(hi);
                    part[e & 1] = add_pair(part[e & 1], pair(lo, hi));
                    pr[e] = round_pair<BF16>(lo, hi);
                }
                tmem_st16(s_cols + 16 * b, pr);
            }
            sum2 = add_pair(sum2, add_pair(part[0], part[1]));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(turn(p_ready, g, j));
        }
        if (ok && n[g] > 0) ok = bar_wait(all_done + 8 * g, 0, stop);
        tc_fence_after();
        float lo, hi;
        unpair(lo, hi, sum2);
        const float sum = lo + hi;
        const bool live = ok && i_row < s.rows && n[g] > 0 && sum > 0.0f;
        if (cut) {
            // A part's row: O, the maximum and the sum as they are.
            float* to = p.part + static_cast<int64_t>(blockIdx.x - p.whole) * h3qk_core::tile_part_floats(p.dim);
            const int tr = g * kTile + r;
            const bool some = i_row < s.rows && n[g] > 0;
            *reinterpret_cast<float2*>(to + 2 * kTile * p.dim + 2 * tr) =
                make_float2(m == -INFINITY ? m : m * c, !ok ? __int_as_float(0x7fc00000) : some ? sum : 0.0f);
#pragma unroll
            for (int d = 0; d < DP; d += 32) {
                uint32_t o[32];
                if (n[g] > 0) {
                    tmem_ld32(o, o_cols + d);
                    tmem_wait_ld(o);
                }
                if (some)
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (d + e < p.dim)
                            *reinterpret_cast<uint4*>(to + tr * p.dim + d + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        const bool write = !cut && i_row < s.span;
        const int64_t row = s.row0 + i_row;
        if (write)
            p.lse[(static_cast<int64_t>(s.item) * p.heads + head) * p.q_rows + row] =
                !ok ? __int_as_float(0x7fc00000)
                    : (i_row < s.rows && n[g] > 0 && !(sum == 0.0f))
                          ? ((m == -INFINITY ? 0.0f : m * c) - kShift + log2f(sum)) * h3qk_core::kLn2
                          : -INFINITY;
        const bool nan_row = ok && i_row < s.rows && n[g] > 0 && sum != sum;
        const float inv = nan_row ? sum : live ? 1.0f / sum : 0.0f;
        uint16_t* out = p.out + s.item * p.os.item + head * p.os.head + row * p.os.row;
#pragma unroll
        for (int d = 0; d < DP; d += 32) {
            uint32_t o[32];
            if (n[g] > 0 && !cut) {
                tmem_ld32(o, o_cols + d);
                tmem_wait_ld(o);
            }
            if (write) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (d + 8 * q < p.dim) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = live || nan_row ? round_pair<BF16>(__uint_as_float(o[8 * q + 2 * e]) * inv,
                                                                      __uint_as_float(o[8 * q + 2 * e + 1]) * inv)
                                                   : 0u;
                        *reinterpret_cast<uint4*>(out + d + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (threadIdx.x == 0 && *stop) atomicAdd(p.stuck, 1u);
    if (warp == 8) {
        tc_fence_after();
        tmem_free(sh.tmem, 512);
    }
}

// One warp a row of a tail tile: its parts' O, weighted to their common
// maximum, in order.
template <bool BF16>
__global__ void __launch_bounds__(256) join_parts_kernel(const __grid_constant__ Params p)
{
    constexpr float kShift = BF16 ? 0.0f : 7.0f;
    h3qk_ops::wait_for_previous();
    const int lane = threadIdx.x & 31, d = 4 * lane;
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), tail = row / (2 * kTile), tr = row % (2 * kTile);
    const Place at = place_of(p, p.whole + tail);
    Stretch s;
    const bool there = h3qk_core::find_stretch(s, p, at.tile, at.item, 2 * kTile, false);
    const int i_row = s.tile * 2 * kTile + tr;
    if (!there || i_row >= s.span) return;
    const int64_t size = h3qk_core::tile_part_floats(p.dim);
    const float* part = p.part + static_cast<int64_t>(tail) * p.parts * size;
    float2 mine = make_float2(-INFINITY, 0.0f);
    if (lane < p.parts) mine = __ldcg(reinterpret_cast<const float2*>(part + lane * size + 2 * kTile * p.dim + 2 * tr));
    if (mine.y == 0.0f) mine.x = -INFINITY;  // no visible key: no O either
    float top = mine.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = mine.y == 0.0f ? 0.0f : exp2_fast(mine.x - top);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < p.parts; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i), li = __shfl_sync(0xffffffffu, mine.y, i);
        sum = fmaf(li, fi, sum);
        if (li != 0.0f && d < p.dim) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + i * size + static_cast<int64_t>(tr) * p.dim + d));
            v.x = fmaf(x.x, fi, v.x);
            v.y = fmaf(x.y, fi, v.y);
            v.z = fmaf(x.z, fi, v.z);
            v.w = fmaf(x.w, fi, v.w);
        }
    }
    const int64_t out_row = s.row0 + i_row;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (d < p.dim) {
        uint2 w;
        w.x = round_pair<BF16>(v.x * inv, v.y * inv);
        w.y = round_pair<BF16>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(p.out + s.item * p.os.item + at.head * p.os.head + out_row * p.os.row + d) = w;
    }
    if (lane == 0)
        p.lse[(static_cast<int64_t>(s.item) * p.heads + at.head) * p.q_rows + out_row] =
            sum == 0.0f ? -INFINITY : (top - kShift + log2f(sum)) * h3qk_core::kLn2;
}

template <bool BF16, int DP, int BENDS>
cudaError_t launch(const Params& p, const h3qk_core::Maps& m, cudaStream_t st)
{
    constexpr int smem = FwdShape<DP>::kSmem;
    auto* kernel = attention_kernel<BF16, DP, BENDS>;
    static bool done[64] = {false};
    const cudaError_t e = h3qk_core::ready(kernel, smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<p.whole + p.tail * p.parts, kThreads, smem, st>>>(m.q, m.k, m.v, p);
    h3qk_internal_count_launch();
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess || p.tail == 0) return launched;
    return h3qk_ops::launch_chained(join_parts_kernel<BF16>, dim3(static_cast<unsigned>(p.tail) * (2 * kTile / 8)), dim3(256), 0,
                                    st, p);
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

cudaError_t h3qk_core::forward_tiles(bool bf16, const Params& p, const Maps& m, cudaStream_t st)
{
    return bf16 ? by_shape<true>(p, m, st) : by_shape<false>(p, m, st);
}
