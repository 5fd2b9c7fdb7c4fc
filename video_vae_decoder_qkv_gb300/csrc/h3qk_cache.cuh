// What the paged cache's kernels share: the pool and its table, how a packed
// row finds its sequence, and the 4-bit format's conversions.
#pragma once

#include "h3qk_ops.cuh"

namespace h3qk_pages {

// The pool and its table.  Strides are in bytes.
struct Pool {
    uint8_t *k, *v, *k_scales, *v_scales;
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;
    int64_t ks_page, ks_head, vs_page, vs_head;
    uint32_t k_page16, v_page16, ks_page16, vs_page16;  // the page strides in pieces of 16 bytes
    const int32_t* table;
    int64_t table_stride;
    const int32_t* kv_lens;
    int32_t pages, max_pages, batch, kv_heads, dim;
    int32_t page_shift;  // log2 of a page's rows
    float k_scale, v_scale;
};

// A sequence's keys, at most what its table has room for.
__device__ __forceinline__ int keys_of(const Pool& c, int item)
{
    return min(max(__ldg(c.kv_lens + item), 0), c.max_pages << c.page_shift);
}

// The page of a sequence's row, or -1 where it has none.
__device__ __forceinline__ int page_of(const Pool& c, const int32_t* row_of_table, int at)
{
    const int n = at >> c.page_shift;
    if (n >= c.max_pages) return -1;
    const int page = __ldg(row_of_table + n);
    return page >= 0 && page < c.pages ? page : -1;
}

// Where a sequence's packed rows lie: [first, first + n).
struct Rows {
    int first, n;
};
__device__ __forceinline__ Rows rows_of(const int32_t* offsets, int each, int tokens, int item)
{
    Rows r;
    if (!offsets) {
        r.first = item * each;
        r.n = each;
    } else {
        r.first = min(max(__ldg(offsets + item), 0), tokens);
        r.n = max(min(__ldg(offsets + item + 1), tokens) - r.first, 0);
    }
    return r;
}

// e2m1: eight codes of a word to four pairs of binary16 (channel 2i low).
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
// Two e4m3 bytes (low 16 bits of w) to a pair of binary16; exact.
__device__ __forceinline__ uint32_t widen_scales(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
    return r;
}
// One half of a pair twice (as moves, which the products take as operand forms).
__device__ __forceinline__ uint32_t both_low(uint32_t a)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t both_high(uint32_t a)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

}  // namespace h3qk_pages
