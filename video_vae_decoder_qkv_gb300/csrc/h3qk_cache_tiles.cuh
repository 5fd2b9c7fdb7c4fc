// Attention over a paged cache, many rows (chunks of prompt): one block takes
// 256 packed rows of a K/V head and streams its keys and values once.
//
// The softmax, the order of the products and the use of TMEM are the dense
// forward kernel's (h3qk_attn_fwd.cu): two groups of four warps own 128 rows
// each, one thread a row, and one warp issues the products of one group while
// the other computes its softmax.  What differs is where rows and keys come
// from:
//  - packed rows: all heads that share a K/V head are in the tile, so keys
//    are loaded (and 4-bit ones converted) once for all of them, and a short
//    chunk's rows still fill a tile.  Rows are not a box of the tensor then:
//    each thread copies its own row into the swizzled tile.
//  - 16-bit pages: one warp loads tiles of 128 keys by TMA, a box for each
//    page (or for 128 rows of a larger one), each lane its own page.
//  - 4-bit pages: three warps copy codes and scales two tiles ahead into
//    shared memory, convert them and store binary16 tiles, swizzled as TMA
//    would: a warp-wide copy is 512 contiguous bytes, each lane converts the 16
//    bytes that it copied, and eight lanes that store together are eight rows
//    of one 16-byte column, which meet no bank twice.  (Ahead in registers,
//    the loads were spilled and waited for one by one.)
//    The products are binary16's whatever the type of q; bfloat16 rows are
//    scaled by a power of two first, as in the kernel for few rows.
//
// Where the tiles are at most half the SMs, each one's keys are shared by
// several blocks, whose results a chained kernel joins in order.  Only the
// device knows how many tiles there are: every block counts them.
#pragma once

#include <type_traits>

#include "h3qk_cache_attn.cuh"

namespace {

using namespace h3qk_tc;
using namespace h3qk_pages;
using h3qk_core::Bend;

constexpr int kTile = 128;              // rows of a group, keys of a tile
constexpr int kThreads = 384;           // 2 x 4 softmax warps; products; three for the keys
constexpr float kSlack = 8.0f;          // log2: growth of the maximum that is tolerated
constexpr int kBlockBytes = 128 * 128;  // 64 columns of a tile

template <bool E2M1, int DP>
struct Shape {
    static constexpr int kBlocks = DP / 64;
    static constexpr int kTileBytes = kBlocks * kBlockBytes;
    static constexpr int kStages = DP == 128 ? (E2M1 ? 4 : 5) : 8;
    static constexpr int kScores = DP == 128 ? 2 : 3;  // S buffers
    static constexpr uint32_t kOut = 128 * kScores;    // first column of O
    // 4 bits: tiles of codes and of scales on their way
    static constexpr int kAhead = 3, kCodes = kTile * DP / 2, kScaleBytes = kTile * DP / 16;
    static constexpr int kCodeStage = kCodes + kScaleBytes;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + (E2M1 ? kAhead * kCodeStage : 0);
};

struct Shared {
    uint64_t full[8], empty[8];
    uint64_t q_full, fixed;
    uint64_t s_full[4], p_ready[4], o_done[2], all_done[2], drain;
    uint32_t tmem;
    int stop;
};

// A block's tile: which sequence, K/V head and 256 packed rows.
struct Place {
    Sequence s;
    int64_t packed;
    int item, kv, tile;
};
__device__ __forceinline__ int64_t packed_of(const Attn& p, const Sequence& s)
{
    const int64_t n = static_cast<int64_t>(s.n) * p.group;
    return n > p.few ? n : 0;
}
__device__ __forceinline__ int64_t tiles_of(const Attn& p, int64_t packed)
{
    return (packed + 2 * kTile - 1) / (2 * kTile) * p.c.kv_heads;
}

// The call's tiles, and how many blocks share the keys of each: as many as
// the SMs have room for, at most kMostParts.
constexpr int kMostParts = 16;
__device__ __forceinline__ int64_t count_tiles(const Attn& p)
{
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int b = lane; b < p.c.batch; b += 32) sum += tiles_of(p, packed_of(p, sequence_of(p, b)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
__device__ __forceinline__ int parts_of(const Attn& p, int64_t tiles)
{
    return tiles > 0 && 2 * tiles <= p.sms ? min(p.sms / static_cast<int>(tiles), kMostParts) : 1;
}
// The tiles of keys that each part takes: four at least, to be worth its own start and the join.
__device__ __forceinline__ int tiles_each(int all, int parts) { return parts == 1 ? all : max((all + parts - 1) / parts, 4); }

// The tile of a block; a sequence's last tiles, which see most, come first, of
// all its K/V heads.
__device__ __forceinline__ void find_place(const Attn& p, int64_t block, Place& at)
{
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int b0 = 0; b0 < p.c.batch; b0 += 32) {
        const int64_t mine = b0 + lane < p.c.batch ? tiles_of(p, packed_of(p, sequence_of(p, b0 + lane))) : 0;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const unsigned vote = __ballot_sync(0xffffffffu, block < before + sum);
        if (vote) {
            const int src = __ffs(vote) - 1;
            before += __shfl_sync(0xffffffffu, sum - mine, src);
            at.item = b0 + src;
            break;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    at.s = sequence_of(p, at.item);
    at.packed = packed_of(p, at.s);
    const int64_t n = block - before, tiles = (at.packed + 2 * kTile - 1) / (2 * kTile);
    at.kv = static_cast<int>(n % p.c.kv_heads);
    at.tile = static_cast<int>(tiles - 1 - n / p.c.kv_heads);
}

// Floats that a part leaves: per row O[dim], then m and sum of every row.
__device__ __forceinline__ int64_t part_floats(int dim) { return h3qk_core::tile_part_floats(dim); }

// E2M1: 4-bit pages, binary16 products; BF16 then only says what q and out are.
template <bool E2M1, bool BF16, int DP, int BENDS>
__global__ void __launch_bounds__(kThreads, 1)
    cache_tiles_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ Attn p)
{
    using S = Shape<E2M1, DP>;
    constexpr int kStages = S::kStages;
    constexpr bool kHalf = E2M1 || !BF16;
    constexpr float kShift = kHalf ? 7.0f : 0.0f;
    constexpr int kLoaders = E2M1 ? 3 : 1;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    h3qk_ops::allow_dependents();
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = base, ring = base + 2 * S::kTileBytes;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int64_t all_tiles = count_tiles(p);
    const int parts = parts_of(p, all_tiles), part = blockIdx.x % parts;
    if (blockIdx.x / parts >= all_tiles) return;
    Place at;
    find_place(p, blockIdx.x / parts, at);
    const Sequence& s = at.s;
    const int64_t tile_row = static_cast<int64_t>(at.tile) * 2 * kTile;
    auto limit = [&](int64_t packed_row) { return limit_of(s, p.causal, static_cast<int>(packed_row / p.group)); };
    int n[2], seen = 0;  // tiles of each group, keys that any row of the block sees
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int64_t first = tile_row + g * kTile;
        const int64_t last = (first + kTile < at.packed ? first + kTile : at.packed) - 1;
        const int lim = last < first ? 0 : limit(last);
        n[g] = (lim + kTile - 1) / kTile;
        seen = max(seen, lim);
    }
    int n_all = max(n[0], n[1]), j0 = 0;  // tiles of this block; the first of them
    if (parts > 1) {
        const int each = tiles_each(n_all, parts), last = n_all;
        j0 = min(part * each, last);
        n_all = min(last - j0, each);
#pragma unroll
        for (int g = 0; g < 2; ++g) n[g] = min(max(n[g] - j0, 0), n_all);
    }
    const int key0 = j0 * kTile;
    // 16-bit pages: V's rows that no row of the block sees are cleared (0 * NaN is NaN, even with p = 0).
    const bool fix = !E2M1 && n_all > 0 && key0 + n_all * kTile > seen;

    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t s_full = smem_addr(sh.s_full), p_ready = smem_addr(sh.p_ready), o_done = smem_addr(sh.o_done);
    const uint32_t all_done = smem_addr(sh.all_done);
    const uint32_t q_full = smem_addr(&sh.q_full), fixed = smem_addr(&sh.fixed);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(full + 8 * i, kLoaders);
            bar_init(empty + 8 * i, 1);
        }
        for (int g = 0; g < 2; ++g) {
            for (int i = 0; i < 2; ++i) {
                bar_init(s_full + 8 * (2 * g + i), 1);
                bar_init(p_ready + 8 * (2 * g + i), 4);
            }
            bar_init(o_done + 8 * g, 1);
            bar_init(all_done + 8 * g, 1);
        }
        bar_init(q_full, 8);
        bar_init(fixed, 1);
        bar_init(smem_addr(&sh.drain), 1);
        sh.stop = 0;
        bar_init_done();
    }
    if (warp == 8) tmem_alloc(smem_addr(&sh.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // the block holds all of TMEM
    volatile int* stop = &sh.stop;
    // A warp's lanes give up together.
    auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_wait(bar, parity, stop)) != 0; };
    auto turn = [](uint32_t bar, int g, int j) { return bar + 8 * (2 * g + (j & 1)); };
    auto phase = [](int j) { return static_cast<uint32_t>(j >> 1) & 1u; };
    const int32_t* table = p.c.table + at.item * p.c.table_stride;
    const int page_mask = (1 << p.c.page_shift) - 1;

    if (warp > 8 && E2M1) {
        regs_down<h3qk_core::kOtherRegs>();
        // ---- 4-bit keys: three warps share a tile's rows ----------------------
        if constexpr (E2M1) {
            constexpr int kPieces = DP / 32;              // 16-byte pieces of codes a row
            constexpr int kRowsEach = 32 / kPieces;       // rows of a warp-wide copy
            constexpr int kTurns = kTile / kRowsEach;     // copies a tile: 16 or 8
            constexpr int kMine = (kTurns + 2) / 3;
            const int w = warp - 9, piece = lane / kRowsEach, sub = lane % kRowsEach;
            const int dim = p.c.dim, row_bytes = dim / 2, groups = dim / 16;
            const bool in = 32 * piece < dim;
            const uint32_t staged = ring + kStages * S::kTileBytes;
            // This lane's 16 bytes of each turn's codes; and of its scales, a few lanes'.
            const int64_t code_at = sub * row_bytes + 16 * piece;
            const bool has_scales = 16 * lane < kRowsEach * groups;
            const uint8_t* codes[2] = {p.c.k + at.kv * p.c.k_head + code_at, p.c.v + at.kv * p.c.v_head + code_at};
            const uint8_t* scales[2] = {p.c.k_scales + at.kv * p.c.ks_head + 16 * lane,
                                        p.c.v_scales + at.kv * p.c.vs_head + 16 * lane};
            auto copy16 = [](uint32_t dst, const uint8_t* src, bool there) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                             : "memory");
            };
            // Copies of tile i (K and V in turn) that fall to this warp.  Lane l
            // holds the page of rows 16 (l mod 8) of the tile's keys.
            int pages = -1;
            auto fetch = [&](int i) {
                if (i < 2 * n_all) {
                    const bool v = i & 1;
                    const int key_tile = key0 + (i >> 1) * kTile;
                    if (!v) {
                        const int key = key_tile + 16 * (lane & 7);
                        pages = key < seen ? page_of(p.c, table, key) : -1;
                    }
                    const uint32_t to = staged + i % S::kAhead * S::kCodeStage;
                    const uint8_t* from = v ? codes[1] : codes[0];
                    const uint8_t* scale_from = v ? scales[1] : scales[0];
                    const int64_t stride = v ? p.c.v_page : p.c.k_page, scale_stride = v ? p.c.vs_page : p.c.ks_page;
#pragma unroll
                    for (int u = 0; u < kMine; ++u) {
                        const int t = (w + i) % 3 + 3 * u;
                        const int page = __shfl_sync(0xffffffffu, pages, t * kRowsEach / 16 & 7);
                        if (t >= kTurns) continue;
                        const int in_page = (key_tile + t * kRowsEach) & page_mask;
                        const bool there = page >= 0;
                        const int64_t pg = there ? page : 0;
                        copy16(to + (t * 32 + lane) * 16, in ? from + pg * stride + in_page * row_bytes : p.c.k, there && in);
                        if (has_scales)
                            copy16(to + S::kCodes + t * kRowsEach * groups + 16 * lane,
                                   scale_from + pg * scale_stride + in_page * groups, there);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            for (int i = 0; i < S::kAhead - 1; ++i) fetch(i);
            const uint32_t store_at = (piece >> 1) * kBlockBytes + sub * 128 + ((((piece & 1) * 4) ^ (sub & 7)) << 4);
            for (int i = 0; i < 2 * n_all; ++i) {
                const int st = i % kStages;
                __syncwarp();  // the codes that are overwritten now have been read
                fetch(i + S::kAhead - 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(S::kAhead - 1) : "memory");
                __syncwarp();
                if (!wait(empty + 8 * st, ((i / kStages) & 1) ^ 1)) break;
                const uint32_t tile = ring + st * S::kTileBytes + store_at, from = staged + i % S::kAhead * S::kCodeStage;
                const int left = seen - (key0 + (i >> 1) * kTile) - sub;  // rows behind it hold nothing
#pragma unroll
                for (int u = 0; u < kMine; ++u) {
                    const int t = (w + i) % 3 + 3 * u;
                    if (t >= kTurns) continue;
                    uint32_t c[4], two = 0;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                                 : "r"(from + (t * 32 + lane) * 16)
                                 : "memory");
                    if (in && t * kRowsEach < left) {
                        uint16_t b;
                        asm volatile("ld.shared.u16 %0, [%1];"
                                     : "=h"(b)
                                     : "r"(from + S::kCodes + (t * kRowsEach + sub) * groups + 2 * piece)
                                     : "memory");
                        two = b;
                    }
                    const uint32_t g = widen_scales(two), lo = __byte_perm(g, g, 0x1010), hi = __byte_perm(g, g, 0x3232);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t v[4];
                        widen_codes(c[e], v);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = mul_half2(v[k], e < 2 ? lo : hi);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"((tile ^ (e << 4)) + t * kRowsEach * 128),
                                     "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                     : "memory");
                    }
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(full + 8 * st);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
        }
    } else if (warp > 9) {
        regs_down<h3qk_core::kOtherRegs>();
    } else if (warp == 9) {
        regs_down<h3qk_core::kOtherRegs>();
        // ---- 16-bit keys: a box a page, a lane a box ---------------------------
        const int boxes = page_mask >= kTile - 1 ? 1 : kTile >> p.c.page_shift;
        const int box_rows = kTile / boxes;
        int issued = 0;
        if (n_all > 0) {
            if (lane == 0) {
                tma_prefetch(&map_k);
                tma_prefetch(&map_v);
            }
            for (int i = 0; i < 2 * n_all; ++i) {
                const int st = i % kStages;
                if (!wait(empty + 8 * st, ((i / kStages) & 1) ^ 1)) break;
                if (lane == 0) bar_expect(full + 8 * st, S::kTileBytes);
                __syncwarp();
                if (lane < boxes) {
                    const int key = key0 + (i >> 1) * kTile + lane * box_rows;
                    int page = key < seen ? page_of(p.c, table, key) : -1;
                    if (page < 0) page = 0x7fffffff;  // past the pool: zeros
                    for (int b = 0; b < S::kBlocks; ++b)
                        tma_load(ring + st * S::kTileBytes + b * kBlockBytes + lane * box_rows * 128, (i & 1) ? &map_v : &map_k,
                                 64 * b, key & page_mask, at.kv, page, full + 8 * st);
                }
                issued = i + 1;
            }
        }
        __syncwarp();
        if (fix) {
            const int i = 2 * n_all - 1, st = i % kStages;
            if (wait(full + 8 * st, (i / kStages) & 1)) {
                const int first = max(seen - key0 - (n_all - 1) * kTile, 0);  // rows to keep
                for (int b = 0; b < S::kBlocks; ++b)
                    for (int o = first * 128 + lane * 16; o < kBlockBytes; o += 512)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         ring + st * S::kTileBytes + b * kBlockBytes + o),
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
            for (int i = max(0, issued - kStages); i < issued; ++i)
                for (int t = 0; t < kMaxTries && !bar_test(full + 8 * (i % kStages), (i / kStages) & 1); ++t) {}
        }
    } else if (warp == 8) {
        regs_down<h3qk_core::kOtherRegs>();
        // ---- matrix products ------------------------------------------------
        if (n_all > 0) {
            constexpr uint32_t shape_s = mma_shape(!kHalf, 128, kTile, false);
            constexpr uint32_t shape_o = mma_shape(!kHalf, 128, DP, true);
            const int steps = (p.c.dim + 15) / 16;
            auto release = [&](int i) {
                if (elect_lane()) mma_commit(empty + 8 * (i % kStages));
                __syncwarp();
            };
            auto loaded = [&](int i) { return wait(full + 8 * (i % kStages), (i / kStages) & 1); };
            auto tile_at = [&](int i) { return ring + (i % kStages) * S::kTileBytes; };
            uint32_t s_next = tmem, p_next = tmem;
            auto move = [&](uint32_t& a) { a = a + 128 == tmem + S::kOut ? tmem : a + 128; };
            auto scores = [&](auto group, int j) {
                constexpr int g = decltype(group)::value;
                if (j >= n_all) return true;
                if (g == 0 && !loaded(2 * j)) return false;
                if (j < n[g]) {
                    const uint64_t a = tile_desc(q_smem + g * S::kTileBytes, 16), b = tile_desc(tile_at(2 * j), 16);
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
                if (g == 0 && fix && j + 1 == n_all && !wait(fixed, 0)) return false;
                if (j < n[g]) {
                    if (!wait(turn(p_ready, g, j), phase(j))) return false;
                    tc_fence_after();
                    const uint64_t b = tile_desc(tile_at(2 * j + 1), kBlockBytes);
                    const uint32_t d = tmem + S::kOut + g * DP;
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
            bool ok = wait(q_full, 0) && scores(g0, 0) && scores(g1, 0);
            if constexpr (S::kScores == 2) {
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
        const int g = warp >> 2;
        const int r = threadIdx.x & 127;
        const int64_t row = tile_row + g * kTile + r;  // packed
        const bool has = row < at.packed;
        const int i_row = static_cast<int>((has ? row : at.packed - 1) / p.group);
        const int head = at.kv * p.group + static_cast<int>((has ? row : 0) % p.group);
        const int64_t token = s.first + i_row;
        // ---- this thread's row of Q into its tile ------------------------------
        float raw = E2M1 ? p.c.k_scale : 1.0f;
        if (n_all > 0) {
            const uint16_t* from = p.q + token * p.q_token + head * p.q_head;
            uint4 v[DP / 8];
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
                v[c] = make_uint4(0, 0, 0, 0);
                if (has && 8 * c < p.c.dim) v[c] = __ldg(reinterpret_cast<const uint4*>(from + 8 * c));
            }
            if constexpr (E2M1 && BF16) {
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < DP / 8; ++c)
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                                 __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
                int e;
                const float up = raise_of(max(top & 0xffffu, top >> 16), e);
                raw *= __int_as_float((127 + e - 141) << 23);
                auto half = [&](uint32_t x) {
                    const float2 f = widen_pair<true>(x);
                    return round_pair<false>(f.x * up, f.y * up);
                };
#pragma unroll
                for (int c = 0; c < DP / 8; ++c) v[c] = make_uint4(half(v[c].x), half(v[c].y), half(v[c].z), half(v[c].w));
            }
#pragma unroll
            for (int c = 0; c < DP / 8; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_smem + g * S::kTileBytes + (c >> 3) * kBlockBytes +
                                                                              r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "r"(v[c].x), "r"(v[c].y), "r"(v[c].z), "r"(v[c].w)
                             : "memory");
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(q_full);
        }
        // ---- softmax: one thread a row ------------------------------------------
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_cols = tmem + S::kOut + g * DP + lanes;
        const int lim = limit_of(s, p.causal, i_row);
        const int lim_first = tile_row + g * kTile < at.packed ? limit(tile_row + g * kTile) : 0;
        const Bend bend = h3qk_pages::bend_of(p, head, raw);
        // Scores to powers of two: the bend gives exponents itself.
        const float c = BENDS != h3qk_core::kPlain ? 1.0f : bend.plain;
        const uint64_t cc = pair(c, c);
        float m = -INFINITY;
        uint64_t sum2 = pair(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < n[g] && ok; ++j) {
            ok = wait(turn(s_full, g, j), phase(j));
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_cols = tmem + (2 * j + g) % S::kScores * 128 + lanes;
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
                    sum2 = mul_pair(sum2, pair(f, f));
                    ok = wait(o_done + 8 * g, (j - 1) & 1);
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
            uint64_t add[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t pr[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float lo, hi;
                    unpair(lo, hi, fma_pair(pair(__uint_as_float(sr[b][2 * e]), __uint_as_float(sr[b][2 * e + 1])), cc, nm));
                    lo = exp2_fast(lo);
                    hi = exp2_fast(hi);
                    add[e & 1] = add_pair(add[e & 1], pair(lo, hi));
                    pr[e] = round_pair<!kHalf>(lo, hi);
                }
                tmem_st16(s_cols + 16 * b, pr);
            }
            sum2 = add_pair(sum2, add_pair(add[0], add[1]));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(turn(p_ready, g, j));
        }
        if (ok && n[g] > 0) ok = wait(all_done + 8 * g, 0);
        tc_fence_after();
        float lo, hi;
        unpair(lo, hi, sum2);
        const float sum = lo + hi;
        const bool some = has && n[g] > 0;
        const bool cut = parts > 1;
        if (cut) {
            // A part's row: O, the maximum and the sum as they are.
            float* to = p.part + static_cast<int64_t>(blockIdx.x) * part_floats(p.c.dim);
            const int tr = g * kTile + r;
            *reinterpret_cast<float2*>(to + 2 * kTile * p.c.dim + 2 * tr) =
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
                        if (d + e < p.c.dim)
                            *reinterpret_cast<uint4*>(to + tr * p.c.dim + d + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        const bool write = !cut && has;
        if (write)
            p.lse[static_cast<int64_t>(head) * p.tokens + token] =
                !ok ? __int_as_float(0x7fc00000)
                    : some && !(sum == 0.0f) ? ((m == -INFINITY ? 0.0f : m * c) - kShift + log2f(sum)) * h3qk_core::kLn2
                                             : -INFINITY;
        const bool nan_row = ok && some && sum != sum, live = ok && some && sum > 0.0f;
        const float inv = nan_row ? sum : live ? (E2M1 ? p.c.v_scale : 1.0f) / sum : 0.0f;
        uint16_t* out = p.out + token * p.out_token + head * p.out_head;
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
                    if (d + 8 * q < p.c.dim) {
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

// One warp a packed row: its parts' O, weighted to their common maximum, in order.
__global__ void __launch_bounds__(256) join_tiles_kernel(const __grid_constant__ Attn p, float shift, float v_scale)
{
    const int lane = threadIdx.x & 31, d = 4 * lane;
    const int64_t block = blockIdx.x / (2 * kTile / 8);
    const int tr = blockIdx.x % (2 * kTile / 8) * 8 + (threadIdx.x >> 5);
    const int64_t all_tiles = count_tiles(p);
    const int parts = parts_of(p, all_tiles);
    if (parts == 1 || block >= all_tiles) return;  // (the tiles wrote their rows themselves)
    Place at;
    find_place(p, block, at);
    h3qk_ops::wait_for_previous();
    const int64_t row = static_cast<int64_t>(at.tile) * 2 * kTile + tr;
    if (row >= at.packed) return;
    const int64_t size = part_floats(p.c.dim);
    const float* part = p.part + block * parts * size;
    float2 mine = make_float2(-INFINITY, 0.0f);
    if (lane < parts) mine = __ldcg(reinterpret_cast<const float2*>(part + lane * size + 2 * kTile * p.c.dim + 2 * tr));
    if (mine.y == 0.0f) mine.x = -INFINITY;  // no visible key: no O either
    float top = mine.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = mine.y == 0.0f ? 0.0f : mine.x == -INFINITY ? 1.0f : exp2_fast(mine.x - top);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < parts; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i), li = __shfl_sync(0xffffffffu, mine.y, i);
        sum = fmaf(li, fi, sum);
        if (li != 0.0f && d < p.c.dim) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part + i * size + static_cast<int64_t>(tr) * p.c.dim + d));
            v.x = fmaf(x.x, fi, v.x);
            v.y = fmaf(x.y, fi, v.y);
            v.z = fmaf(x.z, fi, v.z);
            v.w = fmaf(x.w, fi, v.w);
        }
    }
    finish_row(p, at.s, at.kv, row, d, v, top, sum, shift, v_scale);
}

template <bool E2M1, bool BF16, int DP, int BENDS>
cudaError_t launch(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st)
{
    constexpr int smem = Shape<E2M1, DP>::kSmem;
    auto* kernel = cache_tiles_kernel<E2M1, BF16, DP, BENDS>;
    static bool done[64] = {false};
    const cudaError_t e = h3qk_core::ready(kernel, smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(grid.blocks), kThreads, smem, st>>>(m.k, m.v, p);
    h3qk_internal_count_launch();
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess || grid.join == 0) return launched;
    return h3qk_ops::launch_chained(join_tiles_kernel, dim3(static_cast<unsigned>(grid.join) * (2 * kTile / 8)), dim3(256),
                                    0, st, p, E2M1 || !BF16 ? 7.0f : 0.0f, E2M1 ? p.c.v_scale : 1.0f);
}

// (slopes of 0 where there are none: caps are an instance less that way)
template <bool E2M1, bool BF16, int DP>
cudaError_t by_bends(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st)
{
    using namespace h3qk_core;
    if (p.cap > kWideCap) return launch<E2M1, BF16, DP, kCapped | kSloped | kWide>(p, m, grid, st);
    if (p.cap > 0.0f)
        return p.slopes ? launch<E2M1, BF16, DP, kCapped | kSloped>(p, m, grid, st)
                        : launch<E2M1, BF16, DP, kCapped>(p, m, grid, st);
    return p.slopes ? launch<E2M1, BF16, DP, kSloped>(p, m, grid, st) : launch<E2M1, BF16, DP, kPlain>(p, m, grid, st);
}

template <bool E2M1, bool BF16>
cudaError_t by_shape(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st)
{
    return p.c.dim <= 64 ? by_bends<E2M1, BF16, 64>(p, m, grid, st) : by_bends<E2M1, BF16, 128>(p, m, grid, st);
}

}  // namespace
