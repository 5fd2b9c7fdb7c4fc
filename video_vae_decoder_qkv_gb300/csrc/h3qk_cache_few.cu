// Attention over a paged cache, few rows (tokens and drafts produced one by
// one, over 4-bit or 16-bit pages).
//
// Bound by reading the cache once: 144 bytes a key and K/V head of 128 in
// 4 bits, 512 in 16.  16 bits reach it: 16 uneven caches of up to 32,768 keys
// take 209 us, 6.5 TB/s.  4 bits leave a multiprocessor 6.5 cycles a key and
// head, in which its four schedulers issue some 18 instructions (four
// conversions, five products with scales and P, and what they need): 32 such
// caches take 130 us, 5.5 TB/s, one of 524,288 keys 112 us.  Twelve warps with
// 168 registers each measured better than sixteen with 128 (148 us) or eight
// with 255 (152).  The packed rows of a sequence (its query rows times the
// heads that share a K/V head) form tiles of 8 or 16.
//
// All keys of the call, sequence after sequence, K/V head after head, row tile
// after tile, are one line of units of 64 keys, cut into equal shares, one a
// block: caches of any mix of lengths keep every SM busy to the end.  A
// block's share may hold the end of one run, whole ones, and the beginning of
// another; whole runs are finished in place, and cut ones leave a partial
// result (O, maximum, sum) that a second, chained kernel joins in order.
//
// Short caches of few sequences (a token's latency) take one launch: a cluster
// of kCluster blocks shares a run, and joins its parts through the blocks'
// shared memory.  One token over 4,896 keys, 4 K/V heads of 64: 7.0 us (with
// blocks of three warps 7.6, and then with the line and its join 10.7); over
// 8,192 keys, the most that a table may have room for here, 8.5, and with the
// line over 8,256 11.7.
//
// Inside a share the block's warps take turns of keys in round robin, each
// with its own copies in flight (cp.async into a ring of its own: no barrier
// between warps), its own running maximum, sum and O, and meet in shared
// memory at the end of the run.
//
// The products are the warp-wide 16 x 8 x 16 ones with the keys as rows:
// S^T = K Q^T takes 16 keys x 8 packed rows, O^T += V^T P^T 16 channels x 8
// rows.  (One tcgen05 tile has 128 rows, of which a token's heads would fill
// five.)  The contraction over channels may run in any order, so that a lane
// takes neighbouring channels of its key, and those of O^T likewise.  P^T
// comes out of the softmax with a key a lane group and is turned by two
// 8 x 8 transposes in registers.
//
// 4 bits: e2m1 codes become binary16 in one conversion for two, times their
// group's scale, exactly.  The products are binary16's whatever the type of
// q: bfloat16 rows are first scaled by a power of two so that their largest
// value is near 2^14, which keeps every channel to 2^-39 of that value
// (raise_of), and P is held 2^11 larger.  V's codes of two neighbouring keys are interleaved by
// nibbles before their conversion, which makes the pairs that the product
// takes.
#include <type_traits>

#include "h3qk_cache_attn.cuh"

namespace {

using namespace h3qk_tc;
using namespace h3qk_pages;
using h3qk_core::Bend;

// The maximum serves on while it grows by less than 2^kSlack, and binary16's P
// is held 2^kRaise larger: at most 2^15, and what falls below 2^-14 keeps an
// absolute 2^-36 of the row's largest.
constexpr float kSlack = 4.0f, kRaise = 11.0f;

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, a row's neighbouring pair a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Where a warp's keys come from: one sequence and K/V head.
struct Source {
    const uint4 *k, *v, *ks, *vs;  // the head's rows in page 0, at this lane's first piece
    int end;                       // keys of the run that are looked at
};

// 4-bit pages.  A turn is 32 keys: codes of K and V, DP / 2 bytes a key (of
// which DIM / 2 are copied), and their scales.  Copies run through the rows
// as they lie in memory; the 16-byte pieces are spread over a 128-byte line's
// slots so that the lanes that read K (4 of a key, 8 keys) and V (8 of a key,
// 4 keys) meet no bank twice.  Where a lane copies and reads is fixed but for
// constants, and kept.
template <int DIM, int NB>
struct Codes {
    static constexpr bool kE2m1 = true;
    static constexpr int DP = DIM <= 64 ? 64 : 128;
    // Twelve warps an SM either way.  One row block: blocks of four, as a cluster's
    // eight blocks are then the more warps (one token over 4,896 keys: 6.8 us, of
    // three 7.6).  Two row blocks: of three (drafts, 24 caches: 69 us, of four 75).
    static constexpr int kTurn = 32, kWarps = NB == 1 ? 4 : 3, kStages = 3, kBlocks = NB == 1 ? 3 : 4;
    static constexpr int kPitch = DP / 2;
    static constexpr int kGroups = DIM / 16;            // scale bytes a row
    static constexpr int kScales = 2 * kTurn * kPitch;  // where the scales begin; V's follow K's
    static constexpr int kStage = kScales + 2 * kTurn * (DP / 16);

    int copy_to, copy_from;    // this lane's first piece: in a stage, in memory (bytes of a row of pieces)
    int scale_to, scale_from;  // its piece of scales
    int k_at, v_at, ks_at, vs_at;
    bool copies, copies_scales, k_in;

    __device__ static int slot(int row, int piece)
    {
        if constexpr (DP == 128) return row / 2 * 128 + ((((row & 1) * 4 + piece) ^ ((row >> 1 & 3) * 2)) * 16);
        else return row / 4 * 128 + ((((row & 3) * 2 + piece) ^ ((row >> 2 & 1) * 2)) * 16);
    }
    static constexpr int kPieces = DP / 32, kRowsEach = 32 / kPieces;  // pieces a row; rows of a warp-wide copy

    __device__ Codes(const Pool&, int lane)
    {
        const int g = lane >> 2, c = lane & 3, row = lane / kPieces, piece = lane % kPieces;
        copies = 32 * piece < DIM;
        copy_to = slot(row, piece);
        copy_from = row * (DIM / 2) + 16 * piece;
        // 16 rows' scales lie together, DIM bytes: lanes 0-7 and 8-15 take K's two halves, 16-31 V's
        copies_scales = 16 * (lane & 7) < DIM;
        scale_to = kScales + (lane >> 4) * kTurn * (DP / 16) + (lane >> 3 & 1) * DP + 16 * (lane & 7);
        scale_from = 16 * (lane & 7);
        k_in = DP / 4 * c < DIM;
        k_at = DP == 128 ? slot(g, c) : slot(g, c >> 1) + 8 * (c & 1);
        v_at = kTurn * kPitch + (DP == 128 ? slot(2 * c, g >> 1) + 8 * (g & 1) : slot(2 * c, g >> 2) + 4 * (g & 3));
        ks_at = kScales + g * kGroups + (DP == 128 ? 2 * c : c);
        vs_at = kScales + kTurn * (DP / 16) + 2 * c * kGroups + (DP == 128 ? g : g >> 1);
    }
    // The channel where piece i of 8 of a lane's share of a Q row begins.
    __device__ static int k_channel(int c, int i) { return DP / 4 * c + 8 * i; }
    // The channel of rows g and g + 8 of product m of O^T: this and the next.
    __device__ static int v_channel(int g, int m) { return DP / 8 * g + 2 * m; }

    __device__ void fetch(const Pool& c, const Source& s, uint32_t to, int j, const int (&page)[2], int lane) const
    {
        const int mask = (1 << c.page_shift) - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool there = page[h] >= 0;
            const uint32_t pg = there ? page[h] : 0;
            const int in_page = (j + 16 * h) & mask;
            const uint8_t* k = reinterpret_cast<const uint8_t*>(s.k + static_cast<uint64_t>(pg) * c.k_page16) + in_page * (DIM / 2) + copy_from;
            const uint8_t* v = reinterpret_cast<const uint8_t*>(s.v + static_cast<uint64_t>(pg) * c.v_page16) + in_page * (DIM / 2) + copy_from;
            if (DIM == DP || copies) {
#pragma unroll
                for (int i = 0; i < 16 / kRowsEach; ++i) {
                    const int dst = (h * 16 + i * kRowsEach) * kPitch;
                    copy16(to + copy_to + dst, k + i * kRowsEach * (DIM / 2), there);
                    copy16(to + copy_to + dst + kTurn * kPitch, v + i * kRowsEach * (DIM / 2), there);
                }
            }
        }
        const int pick = lane & 8 ? page[1] : page[0];
        const uint32_t pg = pick >= 0 ? pick : 0;
        const int in_page = (j + 2 * (lane & 8)) & mask;
        const uint4* base = lane & 16 ? s.vs + static_cast<uint64_t>(pg) * c.vs_page16 : s.ks + static_cast<uint64_t>(pg) * c.ks_page16;
        if (DIM == 128 || copies_scales)
            copy16(to + scale_to, reinterpret_cast<const uint8_t*>(base) + in_page * kGroups + scale_from, pick >= 0);
    }

    // Rows 16 kb + g and + 8 of K as the products' A, steps of 4 channels a
    // lane, for f(step, a).  EDGE: rows from `left` on hold nothing.
    template <bool EDGE, class F>
    __device__ void keys(uint32_t at, int kb, int g, int left, F&& f) const
    {
        constexpr int kWords = DP / 32;
        uint32_t w[2][kWords], sc[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t from = at + k_at + (16 * kb + 8 * t) * kPitch;
            const uint32_t scales = at + ks_at + kb * DP + 8 * t * kGroups;
            uint32_t two;
            if constexpr (DP == 128) {
                const uint4 v = lds128(from);
                w[t][0] = v.x, w[t][1] = v.y, w[t][2] = v.z, w[t][3] = v.w;
                two = lds16(scales);
            } else {
                const uint2 v = lds64(from);
                w[t][0] = v.x, w[t][1] = v.y;
                two = lds8(scales);
            }
            if (DIM < DP && !k_in) two = 0;
            if (EDGE && 16 * kb + 8 * t + g >= left) two = 0;
            const uint32_t wide = widen_scales(two);
            sc[t][0] = both_low(wide);
            if constexpr (DP == 128) sc[t][1] = both_high(wide);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t v[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                widen_codes(w[t][i], v[t]);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[t][e] = mul_half2(v[t][e], sc[t][i / 2]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t a[4] = {v[0][2 * e], v[1][2 * e], v[0][2 * e + 1], v[1][2 * e + 1]};
                f(2 * i + e, a);
            }
        }
    }

    // Keys 16 kb + {2c, 2c + 1, 2c + 8, 2c + 9} of V as the products' A (channels as rows), for f(m, a).
    template <bool EDGE, class F>
    __device__ void values(uint32_t at, int kb, int c, int left, F&& f) const
    {
        constexpr int kWords = DP / 64;
        uint32_t w[4][kWords], byte[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            // (an odd row's pieces lie where the even one's would with the row's bit of the slot set)
            const uint32_t flip = (t & 1) ? (DP == 128 ? 64 : 32) : 0;
            const uint32_t from = at + ((v_at ^ flip) + (16 * kb + 8 * (t >> 1)) * kPitch);
            byte[t] = lds8(at + vs_at + kb * DP + ((t & 1) + 8 * (t >> 1)) * kGroups);
            if constexpr (DP == 128) {
                const uint2 v = lds64(from);
                w[t][0] = v.x, w[t][1] = v.y;
            } else {
                w[t][0] = lds32(from);
            }
            if (EDGE && 16 * kb + 2 * c + (t & 1) + 8 * (t >> 1) >= left) byte[t] = 0;
        }
        const uint32_t s01 = widen_scales(byte[0] | byte[1] << 8), s23 = widen_scales(byte[2] | byte[3] << 8);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            constexpr uint32_t kLow = 0x0f0f0f0fu;
            uint32_t v[4][4];  // channels 0, 2, 4, 6 and 1, 3, 5, 7 of keys 0, 1; of keys 2, 3
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t x = w[2 * t][i], y = w[2 * t + 1][i];
                widen_codes((x & kLow) | ((y << 4) & ~kLow), v[2 * t]);
                widen_codes(((x >> 4) & kLow) | (y & ~kLow), v[2 * t + 1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a[4] = {mul_half2(v[0][e], s01), mul_half2(v[1][e], s01), mul_half2(v[2][e], s23),
                                       mul_half2(v[3][e], s23)};
                f(4 * i + e, a);
            }
        }
    }
};

// 16-bit pages.  A turn is 16 keys.  Copies run through the rows as they lie
// in memory; a row's 16-byte pieces are turned by the row's number, so that
// the four lanes that read a key's pieces meet no bank twice (V's lanes
// meet at most in pairs).
template <int DP_, int NB>
struct Halves {
    static constexpr bool kE2m1 = false;
    static constexpr int DP = DP_;
    static constexpr int kTurn = 16, kWarps = 4, kStages = 3, kBlocks = 2;
    static constexpr int kPitch = DP * 2, kStage = 2 * kTurn * kPitch;
    static constexpr int kK = DP / 32, kV = DP / 64;  // pieces of a lane's K row and V row
    static constexpr int kPieces = DP / 8, kRowsEach = 32 / kPieces;

    int copy_to[DP == 128 ? 4 : 2];  // by the turn's rows modulo 8
    int64_t from_k, from_v;
    bool copies;

    __device__ static int slot(int row, int piece) { return row * kPitch + ((piece ^ ((row & 1) * 4 + (row >> 1 & 3))) * 16); }

    __device__ Halves(const Pool& c, int lane)
    {
        const int row = lane / kPieces, piece = lane % kPieces;
        copies = 8 * piece < c.dim;
        from_k = row * c.k_row + 16 * piece;
        from_v = row * c.v_row + 16 * piece;
#pragma unroll
        for (int i = 0; i < (DP == 128 ? 4 : 2); ++i) copy_to[i] = slot(i * kRowsEach + row, piece);
    }
    __device__ static int k_channel(int c, int i) { return 8 * (c + 4 * i); }
    __device__ static int v_channel(int g, int m) { return m / 4 * 64 + 8 * g + 2 * (m % 4); }

    __device__ void fetch(const Pool& c, const Source& s, uint32_t to, int j, const int (&page)[2], int lane) const
    {
        constexpr int kEight = 8 / kRowsEach;  // copies of 8 rows
        const uint32_t pg = page[0] >= 0 ? page[0] : 0;
        const bool there = page[0] >= 0 && copies;  // (channels past the last are zeros)
        const int64_t in_page = j & ((1 << c.page_shift) - 1);
        const uint8_t* k = reinterpret_cast<const uint8_t*>(s.k + static_cast<uint64_t>(pg) * c.k_page16) + in_page * c.k_row + from_k;
        const uint8_t* v = reinterpret_cast<const uint8_t*>(s.v + static_cast<uint64_t>(pg) * c.v_page16) + in_page * c.v_row + from_v;
        const int left = s.end - j - lane / kPieces;  // (rows that hold nothing may be NaN: zeros instead)
#pragma unroll
        for (int i = 0; i < kTurn / kRowsEach; ++i) {
            const uint32_t dst = to + copy_to[i % kEight] + i / kEight * 8 * kPitch;
            const bool ok = there && i * kRowsEach < left;
            copy16(dst, k + i * kRowsEach * c.k_row, ok);
            copy16(dst + kTurn * kPitch, v + i * kRowsEach * c.v_row, ok);
        }
    }

    template <bool EDGE, class F>
    __device__ void keys(uint32_t at, int, int g, int, F&& f) const
    {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            const uint32_t from = at + slot(g, c + 4 * i);
            const uint4 x = lds128(from), y = lds128(from + 8 * kPitch);
            const uint32_t a[4] = {x.x, y.x, x.y, y.y}, b[4] = {x.z, y.z, x.w, y.w};
            f(2 * i, a);
            f(2 * i + 1, b);
        }
    }

    template <bool EDGE, class F>
    __device__ void values(uint32_t at, int, int c, int, F&& f) const
    {
        const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            uint4 x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = lds128(at + kTurn * kPitch + slot(2 * c + (t & 1), g + 8 * i) + 8 * (t >> 1) * kPitch);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a[4] = {__byte_perm(word(x[0], e), word(x[1], e), 0x5410),
                                       __byte_perm(word(x[0], e), word(x[1], e), 0x7632),
                                       __byte_perm(word(x[2], e), word(x[3], e), 0x5410),
                                       __byte_perm(word(x[2], e), word(x[3], e), 0x7632)};
                f(4 * i + e, a);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// The line of work
// ---------------------------------------------------------------------------
// A sequence's part of the line: `runs` (K/V heads x row tiles) of `per` units.
struct Part {
    Sequence s;
    int packed;  // packed rows
    int tiles, per;
    __device__ int64_t units(const Attn& p) const { return packed ? static_cast<int64_t>(p.c.kv_heads) * tiles * per : 0; }
};
template <int ROWS>
__device__ __forceinline__ Part part_of(const Attn& p, int item)
{
    Part t;
    t.s = sequence_of(p, item);
    t.packed = t.s.n * p.group;
    t.tiles = (t.packed + ROWS - 1) / ROWS;
    t.per = max((t.s.keys + kUnit - 1) / kUnit, 1);  // a row without keys is a unit of its own
    return t;
}

// Warp-wide: all units of the call, and with `place` >= 0 the sequence that
// holds unit `place` and the units before it.
template <int ROWS>
__device__ __forceinline__ int64_t all_units(const Attn& p)
{
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int b = lane; b < p.c.batch; b += 32) sum += part_of<ROWS>(p, b).units(p);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
template <int ROWS>
__device__ __forceinline__ int find_unit(const Attn& p, int64_t place, int64_t& before)
{
    const int lane = threadIdx.x & 31;
    before = 0;
    for (int b0 = 0; b0 < p.c.batch; b0 += 32) {
        const int64_t mine = b0 + lane < p.c.batch ? part_of<ROWS>(p, b0 + lane).units(p) : 0;
        int64_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        const unsigned vote = __ballot_sync(0xffffffffu, place < before + sum);
        if (vote) {
            const int src = __ffs(vote) - 1;
            before += __shfl_sync(0xffffffffu, sum - mine, src);
            return b0 + src;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    return -1;
}
__device__ __forceinline__ int64_t share_of(const Attn& p, int64_t total, int blocks)
{
    const int64_t even = (total + blocks - 1) / blocks;
    return even > p.least ? even : p.least;
}

// A block leaves at most two partial results: of the run that its share
// begins in the middle of (or fills), and of the one that it breaks off.
__host__ __device__ inline int64_t part_floats(int rows, int dim) { return static_cast<int64_t>(rows) * (dim + 2); }

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this block's shared memory in block `rank` of the cluster.
__device__ __forceinline__ uint32_t of_block(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// HALF: the products are binary16's.  BENT: scores are capped, or less a slope times the distance.
template <class T, bool HALF, bool BENT, int NB>
__global__ void __launch_bounds__(32 * T::kWarps, T::kBlocks) few_kernel(const __grid_constant__ Attn p)
{
    constexpr int ROWS = 8 * NB, DP = T::DP;
    constexpr int kWarps = T::kWarps, KB = T::kTurn / 16, kSteps = DP / 16, kOut = DP / 16;
    constexpr float kShift = HALF ? kRaise : 0.0f;
    static_assert(T::kWarps * T::kStages * T::kStage >= kWarps * ROWS * (DP + 4) * 4, "the warps' O fits the rings");
    extern __shared__ __align__(128) uint8_t dynamic[];
    __shared__ float sh_m[kWarps][ROWS], sh_l[kWarps][ROWS];
    __shared__ uint2 sh_q[NB == 1 ? 1 : NB][NB == 1 ? 1 : kSteps][32];  // Q of several blocks, as the products take it
    static_assert(NB <= kWarps, "a warp a block of rows of Q");
    h3qk_ops::allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 3, g = lane >> 2;
    [[maybe_unused]] const uint32_t q_at = smem_addr(&sh_q[0][0][NB == 1 ? 0 : lane]);
    const uint32_t ring = smem_addr(dynamic) + warp * T::kStages * T::kStage;
    float(*sh_o)[ROWS][DP + 4] = reinterpret_cast<float(*)[ROWS][DP + 4]>(dynamic);
    const T format(p.c, lane);

    int64_t begin = 0, end = 1, before = 0;
    int item;
    Part part;
    if (p.cluster) {
        item = blockIdx.x / (kCluster * p.c.kv_heads * p.cluster);
        part = part_of<ROWS>(p, item);
        if (static_cast<int>(blockIdx.x / kCluster % p.cluster) >= part.tiles) return;  // the whole cluster
    } else {
        const int64_t total = all_units<ROWS>(p), share = share_of(p, total, gridDim.x);
        begin = blockIdx.x * share;
        end = min(begin + share, total);
        if (begin >= end) return;
        item = find_unit<ROWS>(p, begin, before);
        part = part_of<ROWS>(p, item);
    }

    for (int64_t pos = begin; pos < end;) {
        int unit, units, kv, row_tile;
        if (p.cluster) {
            const int run = blockIdx.x / kCluster, each = (part.per + kCluster - 1) / kCluster;
            row_tile = run % p.cluster;
            kv = run / p.cluster % p.c.kv_heads;
            unit = min(static_cast<int>(blockIdx.x % kCluster) * each, part.per);
            units = min(part.per - unit, each);
            pos = end;
        } else {
            while (pos >= before + part.units(p)) {  // (every unit up to `end` has a sequence)
                before += part.units(p);
                part = part_of<ROWS>(p, ++item);
            }
            const int64_t run = (pos - before) / part.per;
            unit = static_cast<int>((pos - before) - run * part.per);
            units = static_cast<int>(min(static_cast<int64_t>(part.per - unit), end - pos));
            kv = static_cast<int>(run / part.tiles);
            row_tile = static_cast<int>(run % part.tiles);
            pos += units;
        }
        const Sequence& s = part.s;

        // This lane's packed row of each block of 8 for Q, and the two whose scores it holds.
        float o[kOut][NB][4], m[NB][2], l[NB][2];
        float in[NB][2];
        [[maybe_unused]] float slope[NB][2];
        [[maybe_unused]] int at[NB][2];
        int lim[NB][2], most = 0, least = 1 << 30;  // rows that are none see everything: nobody reads them
        [[maybe_unused]] uint32_t q1[2 * kSteps];  // Q of one block stays in registers
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t q[2 * kSteps];
            const int r = row_tile * ROWS + 8 * b + g;
            const bool has = r < part.packed;
            const int i = has ? divide(r, p.group) : 0, head = kv * p.group + (has ? r - i * p.group : 0);
            const uint16_t* from = p.q + (s.first + i) * p.q_token + head * p.q_head;
#pragma unroll
            for (int e = 0; e < kSteps / 2; ++e) {
                const int channel = T::k_channel(c, e);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (has && channel < p.c.dim) v = __ldg(reinterpret_cast<const uint4*>(from + channel));
                q[4 * e] = v.x, q[4 * e + 1] = v.y, q[4 * e + 2] = v.z, q[4 * e + 3] = v.w;
            }
            float raw = 1.0f;
            if constexpr (T::kE2m1) {
                raw = p.c.k_scale;
                if (p.bf16) {
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 2 * kSteps; ++e) top = __vmaxu2(top, q[e] & 0x7fff7fffu);
                    top = max(top & 0xffffu, top >> 16);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    int e;
                    const float up = raise_of(top, e);
                    raw *= __int_as_float((127 + e - 141) << 23);
#pragma unroll
                    for (int k = 0; k < 2 * kSteps; ++k) {
                        const float2 f = widen_pair<true>(q[k]);
                        q[k] = round_pair<false>(f.x * up, f.y * up);
                    }
                }
            }
            if constexpr (NB == 1) {
#pragma unroll
                for (int k = 0; k < 2 * kSteps; ++k) q1[k] = q[k];
            } else if (warp == b) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) sh_q[b][k][lane] = make_uint2(q[2 * k], q[2 * k + 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int src = (2 * c + h) * 4;
                const float raw_of = __shfl_sync(0xffffffffu, raw, src);
                const int i_of = __shfl_sync(0xffffffffu, i, src), head_of = __shfl_sync(0xffffffffu, head, src);
                const bool has_of = __shfl_sync(0xffffffffu, static_cast<int>(has), src) != 0;
                const Bend bend = h3qk_pages::bend_of(p, head_of, raw_of);
                in[b][h] = bend.in;
                slope[b][h] = bend.slope;
                at[b][h] = s.start + i_of;
                lim[b][h] = 1 << 30;
                if (has_of) {
                    lim[b][h] = limit_of(s, p.causal, i_of);
                    most = max(most, lim[b][h]);
                    least = min(least, lim[b][h]);
                }
                m[b][h] = -INFINITY;
                l[b][h] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kOut; ++k) o[k][b][0] = o[k][b][1] = o[k][b][2] = o[k][b][3] = 0.0f;
        }
#pragma unroll
        for (int e = 1; e < 4; e <<= 1) {
            most = max(most, __shfl_xor_sync(0xffffffffu, most, e));
            least = min(least, __shfl_xor_sync(0xffffffffu, least, e));
        }

        Source src;
        src.k = reinterpret_cast<const uint4*>(p.c.k + kv * p.c.k_head);
        src.v = reinterpret_cast<const uint4*>(p.c.v + kv * p.c.v_head);
        src.ks = reinterpret_cast<const uint4*>(p.c.k_scales + kv * p.c.ks_head);
        src.vs = reinterpret_cast<const uint4*>(p.c.v_scales + kv * p.c.vs_head);
        const int32_t* table = p.c.table + item * p.c.table_stride;
        const int k_first = unit * kUnit;
        src.end = min(k_first + units * kUnit, most);
        constexpr int kStep = T::kTurn * kWarps;

        // The pages of the warp's next turns, one a lane (-1: nothing to read): of
        // 16 turns' two halves, or of 32 turns of 16 keys.
        constexpr int kHalves = T::kTurn / 16, kHeld = 32 / kHalves;
        int pages = -1;
        auto hold = [&](int j) {
            const int key = j + lane / kHalves * kStep + 16 * (lane % kHalves);
            pages = key < src.end ? page_of(p.c, table, key) : -1;
        };
        auto pages_of = [&](int turn, int (&pg)[2]) {
            pg[0] = __shfl_sync(0xffffffffu, pages, turn % kHeld * kHalves);
            pg[1] = kHalves == 2 ? __shfl_sync(0xffffffffu, pages, turn % kHeld * kHalves + 1) : -1;
        };

        // One turn's keys, which are in shared memory.  EDGE: some are hidden
        // from some row, or hold nothing.
        auto compute = [&](auto edge, uint32_t here, int j) {
            constexpr bool EDGE = decltype(edge)::value;
            const int left = src.end - j;
            float sc[KB][NB][4];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int b = 0; b < NB; ++b) sc[kb][b][0] = sc[kb][b][1] = sc[kb][b][2] = sc[kb][b][3] = 0.0f;
                format.template keys<EDGE>(here, kb, g, left, [&](int step, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        if constexpr (NB == 1) {
                            mma16<!HALF>(sc[kb][b], a, q1[2 * step], q1[2 * step + 1]);
                        } else {
                            const uint2 w = lds64(q_at + (b * kSteps + step) * 256);
                            mma16<!HALF>(sc[kb][b], a, w.x, w.y);
                        }
                    }
                });
            }
            // BENT: the scores' exponents.  The cap works on four scores at once, which
            // come multiplied with `in`, so that one bend serves them.
            if constexpr (BENT) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // Fours: of one row over two blocks of keys; or of both rows, whose reciprocals
                    // then lie apart (a row's NaN, from its Q or a key that it sees, is not the other's).
                    constexpr bool kApart = KB == 1;
                    float* v[KB][4];
#pragma unroll
                    for (int f = 0; f < KB; ++f)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[f][i] = kApart ? &sc[0][b][i] : &sc[i / 2][b][2 * (i & 1) + f];
                    auto row_of = [](int f, int i) { return kApart ? i & 1 : f; };
                    auto key_of = [&](int i) { return j + (kApart ? 8 * (i / 2) : 16 * (i / 2) + 8 * (i & 1)) + g; };
#pragma unroll
                    for (int f = 0; f < KB; ++f) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int h = row_of(f, i);
                            // (hidden scores may be NaN, and a row's share a reciprocal)
                            if (EDGE && key_of(i) >= lim[b][h]) *v[f][i] = 0.0f;
                            *v[f][i] *= in[b][h];
                        }
                        if (p.cap > 0.0f) {
                            Bend bend;
                            bend.in = 1.0f;
                            bend.plain = 0.5f * p.cap;
                            bend.cap = p.cap * h3qk_core::kLog2e;
                            bend.slope = 0.0f;
                            uint64_t z[2] = {pair(*v[f][0], *v[f][1]), pair(*v[f][2], *v[f][3])}, keep[2];
                            if (p.cap > h3qk_core::kWideCap)
                                h3qk_core::bend_four<h3qk_core::kCapped | h3qk_core::kWide, false, kApart>(z, bend, 0.0f, 0.0f, keep);
                            else
                                h3qk_core::bend_four<h3qk_core::kCapped, false, kApart>(z, bend, 0.0f, 0.0f, keep);
                            unpair(*v[f][0], *v[f][1], z[0]);
                            unpair(*v[f][2], *v[f][3], z[1]);
                        }
                        if (p.slopes)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int h = row_of(f, i);
                                *v[f][i] = fmaf(-slope[b][h], fabsf(static_cast<float>(at[b][h] - key_of(i))), *v[f][i]);
                            }
                    }
                }
            }
            float top[NB][2];  // in powers of two
            bool grows = false;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float t = -INFINITY;
#pragma unroll
                    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& v = sc[kb][b][2 * e + h];
                            if (EDGE) v = j + 16 * kb + 8 * e + g < lim[b][h] ? v : -INFINITY;
                            t = fmaxf(t, v);
                        }
                    top[b][h] = BENT ? t : t * in[b][h];
                    grows = grows || top[b][h] > m[b][h] + kSlack;
                }
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float t = top[b][h];
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
                        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
                        t = fmaxf(t, m[b][h]);
                        const float f = t == -INFINITY ? 1.0f : exp2_fast(m[b][h] - t);
                        m[b][h] = t;
                        l[b][h] *= f;
#pragma unroll
                        for (int k = 0; k < kOut; ++k) {
                            o[k][b][h] *= f;
                            o[k][b][2 + h] *= f;
                        }
                    }
            }
            uint32_t pt[KB][NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float off[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) off[h] = kShift - (m[b][h] == -INFINITY ? 0.0f : m[b][h]);
                auto power = [&](float v, int h) { return exp2_fast(BENT ? v + off[h] : fmaf(v, in[b][h], off[h])); };
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = power(sc[kb][b][2 * e], 0), p1 = power(sc[kb][b][2 * e + 1], 1);
                        l[b][0] += p0;
                        l[b][1] += p1;
                        pt[kb][b][e] = transpose8(round_pair<!HALF>(p0, p1));
                    }
            }
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
                format.template values<EDGE>(here, kb, c, left, [&](int k, const uint32_t (&a)[4]) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) mma16<!HALF>(o[k][b], a, pt[kb][b][0], pt[kb][b][1]);
                });
        };

        if constexpr (NB > 1) __syncthreads();
        const int plain_end = min(src.end, least);
        int j = k_first + T::kTurn * warp;
        if (j < src.end) {
            int pg[2], ahead = 0;  // turns fetched
            hold(j);
#pragma unroll
            for (; ahead < T::kStages - 1; ++ahead) {
                pages_of(ahead, pg);
                if (j + ahead * kStep < src.end) format.fetch(p.c, src, ring + ahead * T::kStage, j + ahead * kStep, pg, lane);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            int stage = 0;
            for (; j < src.end; j += kStep, ++ahead) {
                const int next = j + (T::kStages - 1) * kStep;
                if (ahead % kHeld == 0) hold(next);
                pages_of(ahead, pg);
                __syncwarp();  // the stage that is filled now has been read by all lanes
                if (next < src.end)
                    format.fetch(p.c, src, ring + (stage == 0 ? T::kStages - 1 : stage - 1) * T::kStage, next, pg, lane);
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group %0;" ::"n"(T::kStages - 1) : "memory");
                __syncwarp();
                const uint32_t here = ring + stage * T::kStage;
                stage = stage + 1 == T::kStages ? 0 : stage + 1;
                if (j + T::kTurn <= plain_end) compute(std::false_type{}, here, j);
                else compute(std::true_type{}, here, j);
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        // Join the block's warps.
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = l[b][h];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = 8 * b + 2 * c + h;
                if (g == 0) {
                    sh_m[warp][row] = m[b][h];
                    sh_l[warp][row] = sum;
                }
#pragma unroll
                for (int k = 0; k < kOut; ++k)
                    *reinterpret_cast<float2*>(&sh_o[warp][row][T::v_channel(g, k)]) = make_float2(o[k][b][h], o[k][b][2 + h]);
            }
        __syncthreads();
        const bool whole = units == part.per && !p.cluster;
        // (of a cluster: this block's part, behind the warps' O)
        float* shared_part = reinterpret_cast<float*>(dynamic) + kWarps * ROWS * (DP + 4);
        static_assert(T::kWarps * T::kStages * T::kStage >= (kWarps * ROWS * (DP + 4) + ROWS * (DP + 2)) * 4, "a part fits behind");
        float* to = p.cluster ? shared_part : p.part + (2 * static_cast<int64_t>(blockIdx.x) + (unit == 0 ? 1 : 0)) * part_floats(ROWS, p.c.dim);
        const int per = p.c.dim / 4;
        for (int i = threadIdx.x; i < ROWS * per; i += 32 * kWarps) {
            const int row = i / per, d = 4 * (i - row * per);
            const int r = row_tile * ROWS + row;
            if (r >= part.packed) break;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][row]);
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a warp that saw no key; but a NaN is passed on
                const float f = sh_m[w][row] == -INFINITY ? (sh_l[w][row] == 0.0f ? 0.0f : 1.0f) : exp2_fast(sh_m[w][row] - top);
                const float4 x = *reinterpret_cast<const float4*>(&sh_o[w][row][d]);
                sum = fmaf(sh_l[w][row], f, sum);
                v.x = fmaf(x.x, f, v.x);
                v.y = fmaf(x.y, f, v.y);
                v.z = fmaf(x.z, f, v.z);
                v.w = fmaf(x.w, f, v.w);
            }
            if (whole) {
                finish_row(p, s, kv, r, d, v, top, sum, kShift, T::kE2m1 ? p.c.v_scale : 1.0f);
            } else {
                *reinterpret_cast<float4*>(to + row * p.c.dim + d) = v;
                if (d == 0) *reinterpret_cast<float2*>(to + ROWS * p.c.dim + 2 * row) = make_float2(top, sum);
            }
        }
        if (!p.cluster) {
            __syncthreads();
            continue;
        }
        // Each block joins a share of the values, part by part in order.
        cluster_sync();
        const uint32_t mine = smem_addr(shared_part);
        for (int i = threadIdx.x + 32 * kWarps * static_cast<int>(blockIdx.x % kCluster); i < ROWS * per;
             i += 32 * kWarps * kCluster) {
            const int row = i / per, d = 4 * (i - row * per), r = row_tile * ROWS + row;
            if (r >= part.packed) break;
            float tops[kCluster], sums[kCluster], top = -INFINITY, sum = 0.0f;
            float4 x[kCluster], v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kCluster; ++w) {
                const uint32_t there = of_block(mine, w);
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                             : "=f"(tops[w]), "=f"(sums[w])
                             : "r"(there + (ROWS * p.c.dim + 2 * row) * 4)
                             : "memory");
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x[w].x), "=f"(x[w].y), "=f"(x[w].z), "=f"(x[w].w)
                             : "r"(there + (row * p.c.dim + d) * 4)
                             : "memory");
                top = fmaxf(top, tops[w]);
            }
#pragma unroll
            for (int w = 0; w < kCluster; ++w) {
                const float f = tops[w] == -INFINITY ? (sums[w] == 0.0f ? 0.0f : 1.0f) : exp2_fast(tops[w] - top);
                sum = fmaf(sums[w], f, sum);
                v.x = fmaf(x[w].x, f, v.x);
                v.y = fmaf(x[w].y, f, v.y);
                v.z = fmaf(x[w].z, f, v.z);
                v.w = fmaf(x[w].w, f, v.w);
            }
            finish_row(p, s, kv, r, d, v, top, sum, kShift, T::kE2m1 ? p.c.v_scale : 1.0f);
        }
        cluster_sync();  // no block leaves while another reads its part
    }
}

// One block a packed row of a run that was cut: its warps take the blocks'
// parts in turn, in order, and are joined in order.
constexpr int kJoinWarps = 4;
template <int ROWS>
__global__ void __launch_bounds__(32 * kJoinWarps) join_few_kernel(const __grid_constant__ Attn p, int blocks,
                                                                   unsigned rows, float shift, float v_scale)
{
    __shared__ float4 sh_v[kJoinWarps][32];
    __shared__ float sh_sum[kJoinWarps], sh_top[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = 4 * lane;
    const int r = static_cast<int>(blockIdx.x % rows);  // packed row of the sequence
    const int kv = static_cast<int>(blockIdx.x / rows % p.c.kv_heads), item = static_cast<int>(blockIdx.x / rows / p.c.kv_heads);
    const Part part = part_of<ROWS>(p, item);
    h3qk_ops::wait_for_previous();
    if (r >= part.packed) return;
    // The units before this sequence, and of all.
    int64_t before = 0, total = 0;
    for (int b = lane; b < p.c.batch; b += 32) {
        const int64_t u = part_of<ROWS>(p, b).units(p);
        total += u;
        if (b < item) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    const int64_t share = share_of(p, total, blocks);
    const int64_t u0 = before + (static_cast<int64_t>(kv) * part.tiles + r / ROWS) * part.per, u1 = u0 + part.per;
    const int first = static_cast<int>(u0 / share), last = static_cast<int>((u1 - 1) / share);
    if (first == last) return;  // finished in place
    const int row = r % ROWS, n = last - first + 1;
    const int64_t size = part_floats(ROWS, p.c.dim);
    // the first block's part is the one that it broke off, the others' the one that they began in
    auto slot = [&](int i) { return p.part + (2 * static_cast<int64_t>(first + i) + (i == 0 ? 1 : 0)) * size; };
    auto stat = [&](int i) { return __ldcg(reinterpret_cast<const float2*>(slot(i) + ROWS * p.c.dim + 2 * row)); };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 32 * kJoinWarps) top = fmaxf(top, stat(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, sh_top[w]);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 < n; i0 += 32 * kJoinWarps) {
        const int mine_at = i0 + lane * kJoinWarps + warp;
        float2 mine = make_float2(-INFINITY, 0.0f);
        if (mine_at < n) mine = stat(mine_at);
        const float f = mine.x == -INFINITY ? (mine.y == 0.0f ? 0.0f : 1.0f) : exp2_fast(mine.x - top);
        const int count = min(32, (n - i0 - warp + kJoinWarps - 1) / kJoinWarps);
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i), li = __shfl_sync(0xffffffffu, mine.y, i);
            sum = fmaf(li, fi, sum);
            if (d < p.c.dim) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(slot(i0 + i * kJoinWarps + warp) + row * p.c.dim + d));
                v.x = fmaf(x.x, fi, v.x);
                v.y = fmaf(x.y, fi, v.y);
                v.z = fmaf(x.z, fi, v.z);
                v.w = fmaf(x.w, fi, v.w);
            }
        }
    }
    sh_v[warp][lane] = v;
    if (lane == 0) sh_sum[warp] = sum;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
        const float4 x = sh_v[w][lane];
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
        sum += sh_sum[w];
    }
    finish_row(p, part.s, kv, r, d, v, top, sum, shift, v_scale);
}

template <class T, bool HALF, bool BENT, int NB>
cudaError_t launch(const Attn& p, int blocks, cudaStream_t st)
{
    constexpr int smem = T::kWarps * T::kStages * T::kStage;
    auto* kernel = few_kernel<T, HALF, BENT, NB>;
    static bool raised[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!raised[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        raised[dev] = true;
    }
    if (p.cluster) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(blocks));
        cfg.blockDim = dim3(32 * T::kWarps);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
        h3qk_internal_count_launch();
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    kernel<<<blocks, 32 * T::kWarps, smem, st>>>(p);
    h3qk_internal_count_launch();
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || blocks == 1) return e;
    const int rows = p.max_rows * p.group;
    const dim3 grid(static_cast<unsigned>(rows) * p.c.kv_heads * p.c.batch);
    return h3qk_ops::launch_chained(join_few_kernel<8 * NB>, grid, dim3(32 * kJoinWarps), 0, st, p, blocks,
                                    static_cast<unsigned>(rows), HALF ? kRaise : 0.0f, T::kE2m1 ? p.c.v_scale : 1.0f);
}

template <template <int, int> class T, int DIM, bool HALF>
cudaError_t by_rows(int row_tile, int blocks, const Attn& p, cudaStream_t st)
{
    const bool bent = p.cap > 0.0f || p.slopes;
    if (row_tile == 8)
        return bent ? launch<T<DIM, 1>, HALF, true, 1>(p, blocks, st) : launch<T<DIM, 1>, HALF, false, 1>(p, blocks, st);
    return bent ? launch<T<DIM, 2>, HALF, true, 2>(p, blocks, st) : launch<T<DIM, 2>, HALF, false, 2>(p, blocks, st);
}

template <bool HALF>
cudaError_t halves(int row_tile, int blocks, const Attn& p, cudaStream_t st)
{
    return p.c.dim <= 64 ? by_rows<Halves, 64, HALF>(row_tile, blocks, p, st) : by_rows<Halves, 128, HALF>(row_tile, blocks, p, st);
}

}  // namespace

int64_t h3qk_pages::few_floats(int blocks, int rows, int dim) { return blocks == 1 ? 0 : 2 * blocks * part_floats(rows, dim); }
int h3qk_pages::few_blocks(bool e2m1, int row_tile)
{
    const int an_sm = !e2m1 ? Halves<128, 1>::kBlocks : row_tile == 8 ? Codes<128, 1>::kBlocks : Codes<128, 2>::kBlocks;
    return an_sm * h3qk_internal_sm_count();
}

cudaError_t h3qk_pages::cache_few(bool e2m1, int row_tile, int blocks, const Attn& p, cudaStream_t st)
{
    if (!e2m1) return p.bf16 ? halves<false>(row_tile, blocks, p, st) : halves<true>(row_tile, blocks, p, st);
    switch (p.c.dim) {
    case 32: return by_rows<Codes, 32, true>(row_tile, blocks, p, st);
    case 64: return by_rows<Codes, 64, true>(row_tile, blocks, p, st);
    case 96: return by_rows<Codes, 96, true>(row_tile, blocks, p, st);
    default: return by_rows<Codes, 128, true>(row_tile, blocks, p, st);
    }
}
