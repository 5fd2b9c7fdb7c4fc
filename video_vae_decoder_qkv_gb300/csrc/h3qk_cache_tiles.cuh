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
// The tiles of the call, sequence after sequence, K/V head after head, each as
// many units as it has tiles of 128 keys and kTileCost more, are one line, cut
// into equal shares, one a block: however few tiles there are, and however
// uneven, the SMs finish together.  A tile that is cut leaves a partial result
// (O, maximum, sum) in each of its blocks, and a chained kernel joins them in
// order.  Only the device knows the sequences' rows and keys: a warp of each
// block finds the block's place in the line.
//
// A tile of at most 128 rows is held by both groups, which take its keys in
// turn and join their results from TMEM.
//
// Bound, 16-bit pages: the groups' chains of products and softmax, as in the
// dense kernel.  40 heads on 8 of 128, bf16, 1,024 rows behind 16,384 keys: 237
// us, 1.40 PFLOP/s (the dense kernel's tiles of single heads: 321).  4 bits: the
// same, with the conversions taking issue slots from the softmax: 271 us, 1.23
// PFLOP/s.  Four uneven chunks: 0.67 ms; with the products and barriers alone
// 0.52, with the softmax alone 0.54.  A warp takes whole blocks of 16 rows, which
// lie on one page: their page is looked up once and their scales come in one
// copy (rows dealt out in smaller turns: 0.69).
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
    uint64_t q_full[2], fixed;
    uint64_t s_full[4], p_ready[4], o_done[2], all_done[2], drain;
    uint32_t tmem;
    int stop;
};

// A sequence's part of the line.
struct Run {
    Sequence s;
    int packed;
    int tiles;
};
__device__ __forceinline__ Run run_of(const Attn& p, int item)
{
    Run r;
    r.s = sequence_of(p, item);
    r.packed = r.s.n * p.group;
    r.tiles = (r.packed + 2 * kTile - 1) / (2 * kTile);
    return r;
}
// A tile's units: the tiles of keys that its rows see, behind kTileCost units
// for its rows of Q, the pipeline's start and its result.  (2,048 rows of a
// fresh prompt, where the first tiles see few keys, 40 heads on 8 of 128: 125 us
// with none, 107 with 1, 88 with 3, 83 with 6, 86 with 10; chunks behind long
// caches 746, 750, 734, 723 and 728.)
constexpr int kTileCost = 5;
__device__ __forceinline__ int units_of(const Attn& p, const Run& r, int tile)
{
    const int last = min((tile + 1) * 2 * kTile, r.packed) - 1;
    return (limit_of(r.s, p.causal, divide(last, p.group)) + kTile - 1) / kTile + kTileCost;
}
// Warp-wide: the units of one K/V head of each lane's run.  Runs of many
// tiles are counted by all lanes together.
__device__ __forceinline__ int64_t count_units(const Attn& p, const Run& r)
{
    constexpr int kAlone = 8;
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    if (r.tiles <= kAlone)
        for (int t = 0; t < r.tiles; ++t) sum += units_of(p, r, t);
    for (unsigned many = __ballot_sync(0xffffffffu, r.tiles > kAlone); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        Run q = {};
        q.s.keys = __shfl_sync(0xffffffffu, r.s.keys, src);
        q.s.start = __shfl_sync(0xffffffffu, r.s.start, src);
        q.s.prefix = __shfl_sync(0xffffffffu, r.s.prefix, src);
        q.packed = __shfl_sync(0xffffffffu, r.packed, src);
        q.tiles = __shfl_sync(0xffffffffu, r.tiles, src);
        int64_t part = 0;
        for (int t = lane; t < q.tiles; t += 32) part += units_of(p, q, t);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == src) sum = part;
    }
    return sum;
}

// The call's line, and a warp's place in it.
struct Line {
    int64_t total, share;
    int64_t before;  // units before the tile
    Run run;
    int item, kv, tile, units;

    __device__ __forceinline__ void count(const Attn& p, int blocks)
    {
        const int lane = threadIdx.x & 31;
        total = 0;
        for (int b0 = 0; b0 < p.c.batch; b0 += 32) {
            Run r = {};
            if (b0 + lane < p.c.batch) r = run_of(p, b0 + lane);
            total += count_units(p, r);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        total *= p.c.kv_heads;
        share = (total + blocks - 1) / blocks;
        if (share < p.least) share = p.least;
    }
    // The tile that holds unit `place` (below total).
    __device__ __forceinline__ void find(const Attn& p, int64_t place)
    {
        const int lane = threadIdx.x & 31;
        before = 0;
        int64_t each = 1;  // units of a K/V head
        for (int b0 = 0; b0 < p.c.batch; b0 += 32) {
            Run r = {};
            if (b0 + lane < p.c.batch) r = run_of(p, b0 + lane);
            const int64_t mine = count_units(p, r);
            int64_t sum = mine * p.c.kv_heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const unsigned vote = __ballot_sync(0xffffffffu, place < before + sum);
            if (vote) {
                const int src = __ffs(vote) - 1;
                before += __shfl_sync(0xffffffffu, sum - mine * p.c.kv_heads, src);
                each = __shfl_sync(0xffffffffu, mine, src);
                item = b0 + src;
                break;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
        run = run_of(p, item);
        kv = static_cast<int>((place - before) / each);
        before += kv * each;
        for (int t0 = 0;; t0 += 32) {
            const int mine = t0 + lane < run.tiles ? units_of(p, run, t0 + lane) : 0;
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += up;
            }
            const unsigned vote = __ballot_sync(0xffffffffu, place < before + sum);
            if (vote || t0 + 32 >= run.tiles) {
                const int src = vote ? __ffs(vote) - 1 : 31;
                before += __shfl_sync(0xffffffffu, sum - mine, src);
                units = __shfl_sync(0xffffffffu, mine, src);
                tile = t0 + src;
                return;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    // The next tile, while `place` (which it holds) is below the total.
    __device__ __forceinline__ void next(const Attn& p)
    {
        before += units;
        if (++tile == run.tiles) {
            tile = 0;
            if (++kv == p.c.kv_heads) {
                kv = 0;
                do {
                    ++item;
                    run = run_of(p, item);
                } while (run.tiles == 0 && item + 1 < p.c.batch);
            }
        }
        units = units_of(p, run, tile);
    }
};

// What a block does of one tile: `n_all` tiles of keys from the j0-th on.
struct Piece {
    int row0;               // the tile's first packed row
    int unit0;              // the first of its units
    int j0, n_all, key0;
    int n[2];               // tiles of keys of each group
    int seen;               // keys that any row sees
    bool halved, whole, fix;
    __device__ __forceinline__ Piece(const Attn& p, const Line& at, int64_t pos, int64_t end, bool codes)
    {
        row0 = at.tile * 2 * kTile;
        unit0 = static_cast<int>(pos - at.before);
        const int past_unit = static_cast<int>(min(static_cast<int64_t>(at.units), end - at.before));
        whole = past_unit - unit0 == at.units;
        j0 = max(unit0 - kTileCost, 0);
        n_all = max(past_unit - kTileCost, 0) - j0;
        int full[2];
        seen = 0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int first = row0 + g * kTile, past = min(first + kTile, at.run.packed);
            const int lim = past <= first ? 0 : limit_of(at.run.s, p.causal, divide(past - 1, p.group));
            full[g] = (lim + kTile - 1) / kTile;
            seen = max(seen, lim);
        }
        if (seen == 0) n_all = 0;
        halved = at.run.packed - row0 <= kTile && n_all > 1;
#pragma unroll
        for (int g = 0; g < 2; ++g) n[g] = halved ? (n_all + 1 - g) / 2 : min(max(full[g] - j0, 0), n_all);
        key0 = j0 * kTile;
        // 16-bit pages: V's rows that no row of the block sees are cleared (0 * NaN is NaN, even with p = 0)
        fix = !codes && n_all > 0 && key0 + n_all * kTile > seen;
    }
};

// A thread's row of a piece.
struct Row {
    int64_t token;
    int first, i, head;  // first: the group's first packed row
    bool has;
    __device__ __forceinline__ Row(const Attn& p, const Line& at, const Piece& pc, int g, int r)
    {
        first = pc.row0 + (pc.halved ? 0 : g * kTile);
        has = first + r < at.run.packed;
        const int row = has ? first + r : at.run.packed - 1;
        i = divide(row, p.group);
        head = at.kv * p.group + row - i * p.group;
        token = at.run.s.first + i;
    }
};

// What a block tells the join of the tile that its share breaks off in: `parts`
// blocks from this one on have a part of it (0: none is left to join).
struct Broken {  // kBrokenFloats words
    int parts, first, packed_left, kv, row;  // the sequence's first row; packed rows from the tile's on; the tile's first
};

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
    // (8 x 200 + 4 x 104 = 12 x 168: the converting warps need more than loading ones)
    constexpr int kMathRegs = E2M1 ? 200 : h3qk_core::kMathRegs, kOtherRegs = E2M1 ? 104 : h3qk_core::kOtherRegs;
    static_assert(8 * kMathRegs + 4 * kOtherRegs == 12 * h3qk_core::kLaunchRegs, "the shares are what the launch gave");
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    h3qk_ops::allow_dependents();
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = base, ring = base + 2 * S::kTileBytes;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    // Each warp's place in the line lies in shared memory: in registers it would
    // push out the scores.
    __shared__ Line places[kThreads / 32];
    Line& at = places[warp];
    if (warp == 0) {
        Line here;
        here.count(p, gridDim.x);
        const int64_t place = blockIdx.x * here.share;
        if (place < here.total) here.find(p, place);
        if (lane < kThreads / 32) places[lane] = here;
    }
    __syncthreads();
    const int64_t begin = blockIdx.x * at.share, end = min(begin + at.share, at.total);
    Broken* broken = reinterpret_cast<Broken*>(p.part + 2 * static_cast<int64_t>(gridDim.x) * part_floats(p.c.dim)) + blockIdx.x;
    if (begin >= end) {
        if (threadIdx.x == 0 && gridDim.x > 1) broken->parts = 0;
        return;
    }
    // Moves on to the next tile; the place where that begins.
    auto advance = [&]() {
        int64_t pos = 0;
        __syncwarp();
        if (lane == 0) {
            Line here = at;
            pos = here.before + here.units;
            if (pos < end) {
                here.next(p);
                at = here;
            }
        }
        __syncwarp();
        return __shfl_sync(0xffffffffu, pos, 0);
    };

    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t s_full = smem_addr(sh.s_full), p_ready = smem_addr(sh.p_ready), o_done = smem_addr(sh.o_done);
    const uint32_t all_done = smem_addr(sh.all_done);
    const uint32_t q_full = smem_addr(sh.q_full), fixed = smem_addr(&sh.fixed);
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
            bar_init(q_full + 8 * g, 4);
        }
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
    const int page_mask = (1 << p.c.page_shift) - 1;

    if (warp > 8 && E2M1) {
        regs_down<kOtherRegs>();
        // ---- 4-bit keys: three warps share a tile's rows ----------------------
        if constexpr (E2M1) {
            constexpr int kPieces = DP / 32;              // 16-byte pieces of codes a row
            constexpr int kRowsEach = 32 / kPieces;       // rows of a warp-wide copy
            // A tile is eight blocks of 16 rows (which lie on one page), kPer copies each;
            // the warps take three, three and two of them, in turn.
            constexpr int kPer = 16 / kRowsEach, kMine = 3;
            const int w = warp - 9, piece = lane / kRowsEach, sub = lane % kRowsEach;
            const int dim = p.c.dim, row_bytes = dim / 2, groups = dim / 16;
            const bool in = 32 * piece < dim;
            const uint32_t staged = ring + kStages * S::kTileBytes;
            // This lane's 16 bytes of each copy of codes; and of a block's scales, a few lanes'.
            const int64_t code_at = sub * row_bytes + 16 * piece;
            const bool has_scales = 16 * lane < dim;
            auto copy16 = [](uint32_t dst, const uint8_t* src, bool there) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                             : "memory");
            };
            const uint32_t store_at = (piece >> 1) * kBlockBytes + sub * 128 + ((((piece & 1) * 4) ^ (sub & 7)) << 4);
            int ring_at = 0;  // tiles (K and V in turn) of the pieces before, in whole rounds of the ring
            bool ok = true;
            for (int64_t pos = begin; pos < end && ok; pos = advance()) {
                const Piece pc(p, at, pos, end, true);
                const int32_t* table = p.c.table + at.item * p.c.table_stride;
                const uint8_t* codes[2] = {p.c.k + at.kv * p.c.k_head + code_at, p.c.v + at.kv * p.c.v_head + code_at};
                const uint8_t* scales[2] = {p.c.k_scales + at.kv * p.c.ks_head + 16 * lane,
                                            p.c.v_scales + at.kv * p.c.vs_head + 16 * lane};
                // Copies of tile i (K and V in turn) that fall to this warp.  Lane l
                // holds the page of rows 16 (l mod 8) of the tile's keys.
                int pages = -1;
                auto fetch = [&](int i) {
                    if (i < 2 * pc.n_all) {
                        const bool v = i & 1;
                        const int key_tile = pc.key0 + (i >> 1) * kTile, ri = ring_at + i;
                        if (!v) {
                            const int key = key_tile + 16 * (lane & 7);
                            pages = key < pc.seen ? page_of(p.c, table, key) : -1;
                        }
                        const uint32_t to = staged + ri % S::kAhead * S::kCodeStage;
                        const uint8_t* from = v ? codes[1] : codes[0];
                        const uint8_t* scale_from = v ? scales[1] : scales[0];
                        const int64_t stride = v ? p.c.v_page : p.c.k_page, scale_stride = v ? p.c.vs_page : p.c.ks_page;
                        const int block0 = (w + ri) % 3 * 3;
#pragma unroll
                        for (int u = 0; u < kMine; ++u) {
                            const int block = block0 + u;
                            const int page = __shfl_sync(0xffffffffu, pages, block & 7);
                            if (block >= 8) continue;
                            const int in_page = (key_tile + 16 * block) & page_mask;
                            const bool there = page >= 0;
                            const int64_t pg = there ? page : 0;
                            const uint8_t* rows = in ? from + pg * stride + in_page * row_bytes : p.c.k;
#pragma unroll
                            for (int q = 0; q < kPer; ++q)
                                copy16(to + ((block * kPer + q) * 32 + lane) * 16, in ? rows + q * kRowsEach * row_bytes : p.c.k,
                                       there && in);
                            if (has_scales)
                                copy16(to + S::kCodes + block * dim + 16 * lane,
                                       scale_from + pg * scale_stride + in_page * groups, there);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                };
                for (int i = 0; i < S::kAhead - 1; ++i) fetch(i);
                for (int i = 0; i < 2 * pc.n_all; ++i) {
                    const int ri = ring_at + i, st = ri % kStages;
                    __syncwarp();  // the codes that are overwritten now have been read
                    fetch(i + S::kAhead - 1);
                    asm volatile("cp.async.wait_group %0;" ::"n"(S::kAhead - 1) : "memory");
                    __syncwarp();
                    ok = wait(empty + 8 * st, ((ri / kStages) & 1) ^ 1);
                    if (!ok) break;
                    const uint32_t tile = ring + st * S::kTileBytes + store_at, from = staged + ri % S::kAhead * S::kCodeStage;
                    const int left = pc.seen - (pc.key0 + (i >> 1) * kTile) - sub;  // rows behind it hold nothing
                    const int block0 = (w + ri) % 3 * 3;
                    // (all reads first: one by one, each would be waited for by itself)
                    uint32_t c[kMine * kPer][4], two[kMine * kPer];
#pragma unroll
                    for (int u = 0; u < kMine * kPer; ++u) {
                        const int t = block0 * kPer + u;
                        if (t >= 8 * kPer) continue;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(c[u][0]), "=r"(c[u][1]), "=r"(c[u][2]), "=r"(c[u][3])
                                     : "r"(from + (t * 32 + lane) * 16)
                                     : "memory");
                        uint16_t b;
                        asm volatile("ld.shared.u16 %0, [%1];"
                                     : "=h"(b)
                                     : "r"(from + S::kCodes + (t * kRowsEach + sub) * groups + 2 * piece)
                                     : "memory");
                        two[u] = in && t * kRowsEach < left ? b : 0;
                    }
#pragma unroll
                    for (int u = 0; u < kMine * kPer; ++u) {
                        const int t = block0 * kPer + u;
                        if (t >= 8 * kPer) continue;
                        const uint32_t g = widen_scales(two[u]), lo = both_low(g), hi = both_high(g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t v[4];
                            widen_codes(c[u][e], v);
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
                for (ring_at += 2 * pc.n_all; ring_at % kStages != 0 && ok; ++ring_at) {
                    ok = wait(empty + 8 * (ring_at % kStages), ((ring_at / kStages) & 1) ^ 1);
                    if (lane == 0) bar_arrive(full + 8 * (ring_at % kStages));
                }
            }
        }
    } else if (warp > 9) {
        regs_down<kOtherRegs>();
    } else if (warp == 9) {
        regs_down<kOtherRegs>();
        // ---- 16-bit keys: a box a page, a lane a box ---------------------------
        const int boxes = page_mask >= kTile - 1 ? 1 : kTile >> p.c.page_shift;
        const int box_rows = kTile / boxes;
        int ring_at = 0, issued = 0, last_fix = -1;
        bool ok = true;
        if (lane == 0) {
            tma_prefetch(&map_k);
            tma_prefetch(&map_v);
        }
        for (int64_t pos = begin; pos < end && ok; pos = advance()) {
            const Piece pc(p, at, pos, end, false);
            const int32_t* table = p.c.table + at.item * p.c.table_stride;
            for (int i = 0; i < 2 * pc.n_all; ++i) {
                const int ri = ring_at + i, st = ri % kStages;
                ok = wait(empty + 8 * st, ((ri / kStages) & 1) ^ 1);
                if (!ok) break;
                if (lane == 0) bar_expect(full + 8 * st, S::kTileBytes);
                __syncwarp();
                if (lane < boxes) {
                    const int key = pc.key0 + (i >> 1) * kTile + lane * box_rows;
                    int page = key < pc.seen ? page_of(p.c, table, key) : -1;
                    if (page < 0) page = 0x7fffffff;  // past the pool: zeros
                    for (int b = 0; b < S::kBlocks; ++b)
                        tma_load(ring + st * S::kTileBytes + b * kBlockBytes + lane * box_rows * 128, (i & 1) ? &map_v : &map_k,
                                 64 * b, key & page_mask, at.kv, page, full + 8 * st);
                }
                issued = ri + 1;
            }
            if (ok && pc.fix) {
                const int ri = ring_at + 2 * pc.n_all - 1, st = ri % kStages;
                ok = wait(full + 8 * st, (ri / kStages) & 1);
                // `fixed` has one phase at a time: the tile that was cleared last has been
                // multiplied (as its stage's next use, where it had one, waited for).
                if (ok && last_fix >= 0 && ri - last_fix < kStages)
                    ok = wait(empty + 8 * (last_fix % kStages), (last_fix / kStages) & 1);
                last_fix = ri;
                if (ok) {
                    const int first = max(pc.seen - pc.key0 - (pc.n_all - 1) * kTile, 0);  // rows to keep
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
            for (ring_at += 2 * pc.n_all; ring_at % kStages != 0 && ok; ++ring_at) {
                ok = wait(empty + 8 * (ring_at % kStages), ((ring_at / kStages) & 1) ^ 1);
                if (lane == 0) bar_arrive(full + 8 * (ring_at % kStages));
                issued = ring_at + 1;
            }
        }
        __syncwarp();
        if (*stop && lane == 0) {
            // Given up: this block's loads must land before it leaves.
            for (int i = max(0, issued - kStages); i < issued; ++i)
                for (int t = 0; t < kMaxTries && !bar_test(full + 8 * (i % kStages), (i / kStages) & 1); ++t) {}
        }
    } else if (warp == 8) {
        regs_down<kOtherRegs>();
        // ---- matrix products ------------------------------------------------
        constexpr uint32_t shape_s = mma_shape(!kHalf, 128, kTile, false);
        constexpr uint32_t shape_o = mma_shape(!kHalf, 128, DP, true);
        const int steps = (p.c.dim + 15) / 16;
        int round = 0, fixes = 0;  // rounds through the ring in the pieces before; cleared tiles
        int done[2] = {0, 0}, rows[2] = {0, 0};  // tiles of the groups in the pieces before; pieces that have any
        bool ok = true;
        for (int64_t pos = begin; pos < end && ok; pos = advance()) {
            const Piece pc(p, at, pos, end, E2M1);
            if (pc.n_all == 0) continue;
            // Each piece begins at the ring's and the S buffers' first, so that the
            // products' operands are made of constants and loop counters: they come
            // from uniform registers.
            auto release = [&](int i) {
                if (elect_lane()) mma_commit(empty + 8 * (i % kStages));
                __syncwarp();
            };
            auto loaded = [&](int i) { return wait(full + 8 * (i % kStages), (i / kStages + round) & 1); };
            auto tile_at = [&](int i) { return ring + (i % kStages) * S::kTileBytes; };
            // The groups take turns.  Both multiply the same tile of keys, which is
            // waited for in group 0's turn and released in group 1's (also where one
            // of them does not use it); or, halved, each its own.
            auto products = [&](auto by_half) {
                constexpr bool H = decltype(by_half)::value;
                const int turns = H ? (pc.n_all + 1) / 2 : pc.n_all;
                uint32_t s_next = tmem, p_next = tmem;
                auto move = [&](uint32_t& a) { a = a + 128 == tmem + S::kOut ? tmem : a + 128; };
                auto scores = [&](auto group, int j) {
                    constexpr int g = decltype(group)::value;
                    if (j >= turns) return true;
                    const int i = H ? 4 * j + 2 * g : 2 * j;
                    const bool mine = j < pc.n[g];
                    if ((H ? mine : g == 0) && !loaded(i)) return false;
                    if (mine) {
                        const uint64_t a = tile_desc(q_smem + g * S::kTileBytes, 16), b = tile_desc(tile_at(i), 16);
                        if (elect_lane()) {
#pragma unroll
                            for (int k = 0; k < DP / 16; ++k)
                                if (k < steps) {
                                    constexpr int kStep = 32 >> 4, kNext = kBlockBytes >> 4;
                                    const uint32_t off = (k >> 2) * kNext + (k & 3) * kStep;
                                    mma_ss(s_next, a + off, b + off, shape_s, k > 0);
                                }
                            mma_commit(turn(s_full, g, done[g] + j));
                        }
                        __syncwarp();
                    }
                    move(s_next);
                    if (H ? mine : g == 1) release(i);
                    return true;
                };
                auto values = [&](auto group, int j) {
                    constexpr int g = decltype(group)::value;
                    const int i = (H ? 4 * j + 2 * g : 2 * j) + 1;
                    const bool mine = j < pc.n[g];
                    if ((H ? mine : g == 0) && !loaded(i)) return false;
                    if ((H ? mine : g == 0) && pc.fix && i + 1 == 2 * pc.n_all && !wait(fixed, fixes & 1)) return false;
                    if (mine) {
                        const int jj = done[g] + j;
                        if (!wait(turn(p_ready, g, jj), phase(jj))) return false;
                        tc_fence_after();
                        const uint64_t b = tile_desc(tile_at(i), kBlockBytes);
                        const uint32_t d = tmem + S::kOut + g * DP;
                        if (elect_lane()) {
#pragma unroll
                            for (int k = 0; k < kTile / 16; ++k)
                                mma_ts(d, p_next + 8 * k, b + (k * 2048 >> 4), shape_o, j > 0 || k > 0);
                            mma_commit((j + 1 < pc.n[g] ? o_done : all_done) + 8 * g);
                        }
                        __syncwarp();
                    }
                    move(p_next);
                    if (H ? mine : g == 1) release(i);
                    return true;
                };
                const std::integral_constant<int, 0> g0;
                const std::integral_constant<int, 1> g1;
                bool go = (pc.n[0] == 0 || wait(q_full, rows[0] & 1)) && scores(g0, 0) &&
                          (pc.n[1] == 0 || wait(q_full + 8, rows[1] & 1)) && scores(g1, 0);
                if constexpr (S::kScores == 2) {
                    for (int j = 0; j < turns && go; ++j)
                        go = values(g0, j) && scores(g0, j + 1) && values(g1, j) && scores(g1, j + 1);
                } else {
                    go = go && scores(g0, 1);
                    for (int j = 0; j < turns && go; ++j)
                        go = values(g0, j) && scores(g1, j + 1) && values(g1, j) && scores(g0, j + 2);
                }
                return go;
            };
            ok = pc.halved ? products(std::true_type{}) : products(std::false_type{});
            // The rest of the round passes empty.
            for (int i = 2 * pc.n_all; i % kStages != 0 && ok; ++i) {
                ok = loaded(i);
                if (lane == 0) bar_arrive(empty + 8 * (i % kStages));
            }
            round += (2 * pc.n_all + kStages - 1) / kStages;
            rows[0] += pc.n[0] > 0;
            rows[1] += pc.n[1] > 0;
            done[0] += pc.n[0];
            done[1] += pc.n[1];
            if (pc.fix) ++fixes;
        }
        __syncwarp();
        if (*stop && elect_lane()) {
            const uint32_t drain = smem_addr(&sh.drain);
            mma_commit(drain);
            for (int t = 0; t < kMaxTries && !bar_test(drain, 0); ++t) {}
        }
        __syncwarp();
    } else {
        regs_up<kMathRegs>();
        const int g = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t o_cols = tmem + S::kOut + g * DP + lanes;
        int done = 0, rescales = 0, ends = 0;  // of this group in the pieces before: tiles, and commits on o_done and all_done
        bool ok = true;
        // (a warp that has given up still writes its rows, as NaN, and what the join reads)
        for (int64_t pos = begin; pos < end; pos = advance()) {
            // What the loop over the keys needs of the piece; the rest is found again
            // behind it (in registers it would push out the scores).
            int n, key_first, key_step, lim, lim_first, place;
            Bend bend;
            {
                const Piece pc(p, at, pos, end, E2M1);
                const Row row(p, at, pc, g, r);
                n = ok ? pc.n[g] : 0;
                key_first = pc.key0 + (pc.halved ? g * kTile : 0);
                key_step = pc.halved ? 2 * kTile : kTile;
                lim = limit_of(at.run.s, p.causal, row.i);
                lim_first = row.first < at.run.packed ? limit_of(at.run.s, p.causal, divide(row.first, p.group)) : 0;
                place = at.run.s.start + row.i;
                // ---- this thread's row of Q into its tile (whose last product is done) ----
                float raw = E2M1 ? p.c.k_scale : 1.0f;
                if (n > 0) {
                    const uint16_t* from = p.q + row.token * p.q_token + row.head * p.q_head;
                    uint4 v[DP / 8];
#pragma unroll
                    for (int c = 0; c < DP / 8; ++c) {
                        v[c] = make_uint4(0, 0, 0, 0);
                        if (row.has && 8 * c < p.c.dim) v[c] = __ldg(reinterpret_cast<const uint4*>(from + 8 * c));
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
                        for (int c = 0; c < DP / 8; ++c)
                            v[c] = make_uint4(half(v[c].x), half(v[c].y), half(v[c].z), half(v[c].w));
                    }
#pragma unroll
                    for (int c = 0; c < DP / 8; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(q_smem + g * S::kTileBytes +
                                                                                      (c >> 3) * kBlockBytes + r * 128 +
                                                                                      (((c & 7) ^ (r & 7)) << 4)),
                                     "r"(v[c].x), "r"(v[c].y), "r"(v[c].z), "r"(v[c].w)
                                     : "memory");
                    fence_async();
                    __syncwarp();
                    if (lane == 0) bar_arrive(q_full + 8 * g);
                }
                bend = h3qk_pages::bend_of(p, row.head, raw);
            }
            // ---- softmax: one thread a row ----------------------------------------
            // Scores to powers of two: the bend gives exponents itself.
            const float c = BENDS != h3qk_core::kPlain ? 1.0f : bend.plain;
            const uint64_t cc = pair(c, c);
            float m = -INFINITY;
            uint64_t sum2 = pair(0.0f, 0.0f);
            for (int j = 0; j < n; ++j) {
                const int jj = done + j, key = key_first + j * key_step;
                ok = wait(turn(s_full, g, jj), phase(jj));
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_cols = tmem + (2 * j + g) % S::kScores * 128 + lanes;
                uint32_t sr[4][32];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld32(sr[b], s_cols + 32 * b);
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_wait_ld(sr[b]);
                const bool edge = key + kTile > lim_first;  // some row sees the tile only in part
                const int left = lim - key;
                auto hide = [&](int b, int e, uint32_t as) {
                    if (32 * b + e >= left) sr[b][e] = as;
                };
                auto bend_all = [&](auto at_edge) {
                    const float far = static_cast<float>(place - key);
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
                    for (int e = 2; e < 32; e += 2)
                        mx[b] = max3(mx[b], __uint_as_float(sr[b][e]), __uint_as_float(sr[b][e + 1]));
                }
                const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                if (__any_sync(0xffffffffu, (top - m) * c > kSlack)) {
                    if (j > 0) {
                        const float f = top == -INFINITY ? 1.0f : exp2_fast((m - top) * c);
                        sum2 = mul_pair(sum2, pair(f, f));
                        // (This S being done, all O but the last one are.)
                        ok = wait(o_done + 8 * g, (rescales + j - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        // (a few columns at a time: the scores fill the registers)
#pragma unroll 1
                        for (int d = 0; d < DP; d += 8) {
                            uint32_t o[8];
                            tmem_ld8(o, o_cols + d);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st8(o_cols + d, o);
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
                        unpair(lo, hi,
                               fma_pair(pair(__uint_as_float(sr[b][2 * e]), __uint_as_float(sr[b][2 * e + 1])), cc, nm));
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
                if (lane == 0) bar_arrive(turn(p_ready, g, jj));
            }
            if (ok && n > 0) ok = wait(all_done + 8 * g, ends & 1);
            tc_fence_after();
            done += n;
            if (n > 0) {
                rescales += n - 1;
                ++ends;
            }

            // ---- this row's result ---------------------------------------------------
            const Piece pc(p, at, pos, end, E2M1);
            const Row row(p, at, pc, g, r);
            float lo, hi;
            unpair(lo, hi, sum2);
            float sum = !ok ? __int_as_float(0x7fc00000) : n > 0 ? lo + hi : 0.0f;
            float top = n > 0 && m != -INFINITY ? m * c : -INFINITY, f0 = 1.0f, f1 = 0.0f;
            if (pc.halved) {
                // The second group leaves its statistics (where its rows of Q were), the
                // first joins both O.
                float2* half = reinterpret_cast<float2*>(smem_raw + (q_smem + S::kTileBytes - smem_addr(smem_raw)));
                if (g == 1) half[r] = make_float2(top, sum);
                tc_fence_before();
                asm volatile("bar.sync 1, 256;" ::: "memory");
                tc_fence_after();
                if (g == 0) {
                    const float2 other = half[r];
                    const float both = fmaxf(top, other.x);
                    f0 = top == -INFINITY ? (sum == 0.0f ? 0.0f : 1.0f) : exp2_fast(top - both);
                    f1 = other.x == -INFINITY ? (other.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(other.x - both);
                    sum = sum * f0 + other.y * f1;
                    top = both;
                }
            }
            if (threadIdx.x == 0 && gridDim.x > 1 && at.before + at.units >= end) {
                // The share ends in this tile.  Its parts: this block's and, the shares being
                // equal, as many as the rest takes; a tile that an earlier block broke off is that one's.
                const int64_t rest = at.before + at.units - end;
                broken->parts = rest > 0 && pc.unit0 == 0 ? 1 + static_cast<int>((rest + at.share - 1) / at.share) : 0;
                broken->first = at.run.s.first;
                broken->packed_left = at.run.packed - pc.row0;
                broken->kv = at.kv;
                broken->row = pc.row0;
            }
            const bool writes = row.has && !(pc.halved && g == 1);
            const bool nan_row = sum != sum, some = n > 0;
            float* to = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (pc.unit0 == 0 ? 1 : 0)) * part_floats(p.c.dim);
            const int tr = (pc.halved ? 0 : g * kTile) + r;
            if (writes) {
                if (!pc.whole) *reinterpret_cast<float2*>(to + 2 * kTile * p.c.dim + 2 * tr) = make_float2(top, sum);
                else
                    p.lse[static_cast<int64_t>(row.head) * p.tokens + row.token] =
                        sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) - kShift + log2f(sum)) * h3qk_core::kLn2;
            }
            const float inv = !pc.whole ? 1.0f : nan_row ? sum : sum == 0.0f ? 0.0f : (E2M1 ? p.c.v_scale : 1.0f) / sum;
            f0 *= inv;
            f1 *= inv;
            uint16_t* out = p.out + row.token * p.out_token + row.head * p.out_head;
#pragma unroll
            for (int d = 0; d < DP; d += 32) {
                uint32_t o[32];
                if (some) {
                    tmem_ld32(o, o_cols + d);
                    tmem_wait_ld(o);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = some ? __float_as_uint(__uint_as_float(o[e]) * f0) : 0u;
                if (pc.halved && g == 0) {
                    uint32_t q[32];
                    tmem_ld32(q, o_cols + DP + d);
                    tmem_wait_ld(q);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(q[e]), f1, __uint_as_float(o[e])));
                }
                if (writes && !pc.whole) {
                    // A part's row: O, the maximum and the sum as they are.
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        if (d + e < p.c.dim)
                            *reinterpret_cast<uint4*>(to + tr * p.c.dim + d + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if (writes) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (d + 8 * q < p.c.dim) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = round_pair<BF16>(__uint_as_float(o[8 * q + 2 * e]), __uint_as_float(o[8 * q + 2 * e + 1]));
                            *reinterpret_cast<uint4*>(out + d + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                }
            }
            tc_fence_before();
            // (the second group's O and statistics have been read)
            if (pc.halved) asm volatile("bar.sync 1, 256;" ::: "memory");
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *stop) atomicAdd(p.stuck, 1u);
    if (warp == 8) {
        tc_fence_after();
        tmem_free(sh.tmem, 512);
    }
}

// For each block whose share broke a tile off: a warp takes four packed rows
// at once, their parts' O, weighted to their common maximum, in order.
constexpr int kJoinWarps = 8, kJoinAtOnce = 4, kJoinRows = kJoinWarps * kJoinAtOnce;  // of a block
__global__ void __launch_bounds__(32 * kJoinWarps) join_tiles_kernel(const __grid_constant__ Attn p, int blocks, float shift,
                                                                     float v_scale)
{
    const int lane = threadIdx.x & 31, d = 4 * lane;
    const int first = blockIdx.x / (2 * kTile / kJoinRows);
    const int tr = blockIdx.x % (2 * kTile / kJoinRows) * kJoinRows + (threadIdx.x >> 5) * kJoinAtOnce;
    const int64_t size = part_floats(p.c.dim);
    // (every block waits: what follows this kernel must find the tiles done)
    h3qk_ops::wait_for_previous();
    const int* words = reinterpret_cast<const int*>(reinterpret_cast<const Broken*>(p.part + 2 * blocks * size) + first);
    int word = 0;
    if (lane < 5) word = __ldcg(words + lane);
    const int n = __shfl_sync(0xffffffffu, word, 0), rows = min(__shfl_sync(0xffffffffu, word, 2) - tr, kJoinAtOnce);
    if (rows <= 0 || n == 0) return;
    Sequence s = {};
    s.first = __shfl_sync(0xffffffffu, word, 1);
    const int kv = __shfl_sync(0xffffffffu, word, 3), row = __shfl_sync(0xffffffffu, word, 4) + tr;
    // the first block's part is the one that it broke off, the others' the one that they began in
    auto slot = [&](int i) { return p.part + (2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0)) * size; };
    auto stat = [&](int i, int q) {
        return __ldcg(reinterpret_cast<const float2*>(slot(i) + 2 * kTile * p.c.dim + 2 * (tr + q)));
    };
    float top[kJoinAtOnce], sum[kJoinAtOnce];
    float4 v[kJoinAtOnce];
#pragma unroll
    for (int q = 0; q < kJoinAtOnce; ++q) {
        top[q] = -INFINITY;
        sum[q] = 0.0f;
        v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int i = lane; i < n; i += 32)
#pragma unroll
        for (int q = 0; q < kJoinAtOnce; ++q)
            if (q < rows) top[q] = fmaxf(top[q], stat(i, q).x);
#pragma unroll
    for (int q = 0; q < kJoinAtOnce; ++q)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], o));
    for (int i0 = 0; i0 < n; i0 += 32) {
        float f[kJoinAtOnce], l[kJoinAtOnce];
#pragma unroll
        for (int q = 0; q < kJoinAtOnce; ++q) {
            float2 mine = make_float2(-INFINITY, 0.0f);
            if (i0 + lane < n && q < rows) mine = stat(i0 + lane, q);
            f[q] = mine.x == -INFINITY ? (mine.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(mine.x - top[q]);
            l[q] = mine.y;
        }
        const int count = min(32, n - i0);
#pragma unroll 2
        for (int i = 0; i < count; ++i)
#pragma unroll
            for (int q = 0; q < kJoinAtOnce; ++q) {
                const float fi = __shfl_sync(0xffffffffu, f[q], i), li = __shfl_sync(0xffffffffu, l[q], i);
                sum[q] = fmaf(li, fi, sum[q]);
                if (d < p.c.dim && q < rows) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(slot(i0 + i) + (tr + q) * p.c.dim + d));
                    v[q].x = fmaf(x.x, fi, v[q].x);
                    v[q].y = fmaf(x.y, fi, v[q].y);
                    v[q].z = fmaf(x.z, fi, v[q].z);
                    v[q].w = fmaf(x.w, fi, v[q].w);
                }
            }
    }
#pragma unroll
    for (int q = 0; q < kJoinAtOnce; ++q)
        if (q < rows) finish_row(p, s, kv, row + q, d, v[q], top[q], sum[q], shift, v_scale);
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
    if (launched != cudaSuccess || grid.blocks == 1) return launched;
    return h3qk_ops::launch_chained(join_tiles_kernel, dim3(static_cast<unsigned>(grid.blocks - 1) * (2 * kTile / kJoinRows)),
                                    dim3(32 * kJoinWarps), 0, st, p, grid.blocks, E2M1 || !BF16 ? 7.0f : 0.0f, E2M1 ? p.c.v_scale : 1.0f);
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
