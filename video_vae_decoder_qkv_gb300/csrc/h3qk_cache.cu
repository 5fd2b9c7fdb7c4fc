// The paged cache: the checks of a pool, appending prepared rows, and reading
// rows back.  Layout and 4-bit format are described at h3qk_cache in h3qk.h.
#include "h3qk_cache_host.h"
#include "h3qk_kernels.cuh"

namespace {

using namespace h3qk_ops;
using namespace h3qk_pages;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

// ---------------------------------------------------------------------------
// Appending: the forward preparation's arithmetic (qk_row, bit for bit), with
// Q to packed rows and K, V to their places in the pages.
//
// Bound by HBM: each packed row is read once, and Q and the cache's bytes are
// written.  The layout is the preparation's: a lane owns CH chunks of 8
// channels, the LPR lanes of a head row are a power of two, a warp holds
// 32 / LPR consecutive packed rows, finds their sequences by a search in the
// offsets, and their angles, once, and walks a slice of the heads, kAhead head
// rows of copies ahead of itself (in shared memory: loads ahead in
// registers were waited for together).  13,000 rows of 40 + 2 x 8 heads of 128
// in 16 bits: 67 us, 5.7 TB/s; 107 with the rows ahead in registers.
//
// 4 bits: a group of 16 channels is two neighbouring lanes.  The largest
// magnitude of its 16-bit values is an integer maximum of their bits (exact,
// and any infinity or NaN wins it), one exchange joins the lanes, and a lane's
// 8 codes are one 4-byte store.  There the instructions count as much as the
// bytes: 32,640 rows of 40 + 2 x 8 heads of 128 take 172 us, 4.9 TB/s, with three
// issue slots of four in use (in 16 bits 155).
// ---------------------------------------------------------------------------
constexpr int kWarps = 8, kBlocks = 3;  // of a block; of an SM
// Head rows of copies ahead: the 4-bit form's longer arithmetic hides them
// behind less (32,640 rows of 40 + 2 x 8 heads of 128: 172 us with 2, 192 with
// 3; in 16 bits 13,000 rows 70 us with 2, 67 with 3).
constexpr int kAhead4 = 2, kAhead16 = 3;

struct AppendArgs {
    h3qk::Params p;  // the preparation's description of the rows; heads: Q, K and V together
    Pool c;
    const int32_t* offsets;
    int32_t each;         // rows a sequence without offsets
    int32_t q_heads;
    uint16_t* out_q;
    int64_t groups;       // groups of 32 / LPR packed rows
    int32_t slices, slice_heads;
    float to_scale[2];    // 1 / (6 k_scale), 1 / (6 v_scale)
};

// The 4-bit codes of a lane's 8 values (16-bit pairs y) and their group's scale byte.
template <bool BF16>
__device__ __forceinline__ uint32_t encode_group(const uint32_t (&y)[4], float to_scale, float tensor_scale, uint32_t& scale)
{
    uint32_t top = __vmaxu2(__vmaxu2(y[0] & 0x7fff7fffu, y[1] & 0x7fff7fffu),
                            __vmaxu2(y[2] & 0x7fff7fffu, y[3] & 0x7fff7fffu));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top & 0xffffu, top >> 16);
    const float amax = h3qk::widen2<BF16>(top).x;
    uint16_t code;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(code)
        : "f"(0.0f), "f"(fmaxf(__fmul_rn(amax, to_scale), 0x1p-9f)));
    const bool finite = top < (BF16 ? 0x7f80u : 0x7c00u);
    scale = finite ? code : 0x7fu;
    const float g = h3qk::widen2<false>(widen_scales(code)).x;
    const float factor = __frcp_rn(__fmul_rn(g, tensor_scale));
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = h3qk::mul2(h3qk::widen2<BF16>(y[i]), make_float2(factor, factor));
        uint32_t byte;
        asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
            : "=r"(byte)
            : "f"(v.y), "f"(v.x));
        codes |= byte << (8 * i);
    }
    return finite ? codes : 0u;
}

template <bool BF16, int LPR, int CH, bool E2M1>
__global__ void __launch_bounds__(32 * kWarps, kBlocks) append_kernel(const __grid_constant__ AppendArgs a)
{
    const h3qk::Params& p = a.p;
    const Pool& c = a.c;
    constexpr int TPW = 32 / LPR, kAhead = E2M1 ? kAhead4 : kAhead16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = lane % LPR, sub = lane / LPR;  // this lane's chunks: chunk + q LPR
    const int D = p.head_dim;
    const int kv_heads = c.kv_heads, q_heads = a.q_heads;
    __shared__ uint4 slots[kWarps][kAhead][CH][32];
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(&slots[warp][0][0][lane]));
    bool in[CH];
#pragma unroll
    for (int q = 0; q < CH; ++q) in[q] = chunk + q * LPR < p.chunks;
    const int64_t items = a.groups * a.slices;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + warp; it < items;
         it += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t group = it / a.slices;
        const int h0 = static_cast<int>(it - group * a.slices) * a.slice_heads;
        const int h1 = min(h0 + a.slice_heads, p.heads);
        const int64_t r = group * TPW + sub;
        const uint16_t* x = p.qkv + r * p.row_stride + 8 * chunk;
        // The row's sequence: the last one whose first row is not behind it
        // (an empty sequence before it starts at the same row).
        int item = -1, start = 0, n = 0;
        if (r < p.rows) {
            if (!a.offsets) {
                item = static_cast<int>(r / a.each);
            } else {
                int lo = 0, hi = c.batch;  // offsets[lo] <= r, or lo = 0
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (__ldg(a.offsets + mid) <= r) lo = mid;
                    else hi = mid;
                }
                item = lo;
            }
            const Rows rows = rows_of(a.offsets, a.each, static_cast<int>(p.rows), item);
            start = rows.first;
            n = rows.n;
        }
        const bool row = item >= 0 && r >= start && r < start + n;
        // (a lane reads back what it copied itself: there is nothing to synchronise)
        auto fetch = [&](int h) {
#pragma unroll
            for (int q = 0; q < CH; ++q) {
                const bool there = row && in[q] && h < h1;
                const uint16_t* from = there ? x + static_cast<int64_t>(h) * D + 8 * q * LPR : p.qkv;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 ring + ((h - h0) % kAhead * CH + q) * 512),
                             "l"(from), "r"(there ? 16 : 0)
                             : "memory");
            }
            h3qk::cp_async_commit();
        };
#pragma unroll
        for (int u = 0; u < kAhead - 1; ++u) fetch(h0 + u);
        int at = 0, page = -1;
        if (row) {
            // (places stay below the length; a negative one's difference is taken in 64 bits)
            const int64_t place = static_cast<int64_t>(__ldg(c.kv_lens + item)) - n + (r - start);
            at = static_cast<int>(max(place, static_cast<int64_t>(INT32_MIN)));
            if (at >= 0) page = page_of(c, c.table + item * c.table_stride, at);
        }
        const int in_page = at & ((1 << c.page_shift) - 1);
        float cs[CH][4], sn[CH][4];
        bool rot[CH][4];
#pragma unroll
        for (int q = 0; q < CH; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cs[q][i] = 1.0f;
                sn[q][i] = 0.0f;
                const int pair = 4 * (chunk + q * LPR) + i;
                rot[q][i] = row && 2 * pair < p.rotary_dim;
                if (rot[q][i] && h0 < q_heads + kv_heads) {
                    const float pos = static_cast<float>(p.pos ? __ldg(p.pos + r * p.n_axes + p.axis[pair]) : at);
                    h3qk::sincos_h3(__fmul_rn(pos, p.inv_freq[pair]), sn[q][i], cs[q][i]);
                }
            }
        // Where this lane's first chunk of K and V head rows goes.
        constexpr int kChunkBytes = E2M1 ? 4 : 16;
        uint8_t* k_to = c.k + (page * c.k_page + in_page * c.k_row + chunk * kChunkBytes);
        uint8_t* v_to = c.v + (page * c.v_page + in_page * c.v_row + chunk * kChunkBytes);
        uint8_t *ks_to = nullptr, *vs_to = nullptr;
        if constexpr (E2M1) {
            ks_to = c.k_scales + (page * c.ks_page + static_cast<int64_t>(in_page) * (D / 16) + chunk / 2);
            vs_to = c.v_scales + (page * c.vs_page + static_cast<int64_t>(in_page) * (D / 16) + chunk / 2);
        }
        uint16_t* out = a.out_q + r * q_heads * D + 8 * chunk;
        const bool placed = row && page >= 0;
        float4 w[2 * CH];
        for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int head = h + u;
                if (head >= h1) break;
                fetch(head + kAhead - 1);
                h3qk::cp_async_wait<kAhead - 1>();
                uint4 raw[CH];
#pragma unroll
                for (int q = 0; q < CH; ++q)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(raw[q].x), "=r"(raw[q].y), "=r"(raw[q].z), "=r"(raw[q].w)
                                 : "r"(ring + (u * CH + q) * 512)
                                 : "memory");
                const bool is_v = head >= q_heads + kv_heads;
                uint32_t y[CH][4];
                if (!is_v) {
                    if (head == h0 || head == q_heads) {
                        const float* from = (head < q_heads ? p.wq : p.wk) + 8 * chunk;
#pragma unroll
                        for (int q = 0; q < CH; ++q)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                w[2 * q + i] = in[q] ? __ldg(reinterpret_cast<const float4*>(from + 8 * q * LPR) + i)
                                                     : make_float4(0, 0, 0, 0);
                    }
                    h3qk::qk_row<BF16, LPR, CH>(raw, w, cs, sn, rot, p.inv_d, p.eps, D, y);
                } else {
#pragma unroll
                    for (int q = 0; q < CH; ++q) y[q][0] = raw[q].x, y[q][1] = raw[q].y, y[q][2] = raw[q].z, y[q][3] = raw[q].w;
                }
                if (head < q_heads) {
#pragma unroll
                    for (int q = 0; q < CH; ++q)
                        if (row && in[q])
                            __stcs(reinterpret_cast<uint4*>(out + static_cast<int64_t>(head) * D + 8 * q * LPR),
                                   make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]));
                    continue;
                }
                const int kv = is_v ? head - q_heads - kv_heads : head - q_heads;
                uint8_t* to = is_v ? v_to + kv * c.v_head : k_to + kv * c.k_head;
                [[maybe_unused]] uint8_t* scale_to = nullptr;
                if constexpr (E2M1) scale_to = is_v ? vs_to + kv * c.vs_head : ks_to + kv * c.ks_head;
#pragma unroll
                for (int q = 0; q < CH; ++q) {
                    if constexpr (E2M1) {
                        uint32_t scale;
                        const uint32_t codes =
                            encode_group<BF16>(y[q], a.to_scale[is_v ? 1 : 0], is_v ? c.v_scale : c.k_scale, scale);
                        if (placed && in[q]) {
                            *reinterpret_cast<uint32_t*>(to + q * LPR * kChunkBytes) = codes;
                            if ((chunk & 1) == 0) scale_to[q * LPR / 2] = static_cast<uint8_t>(scale);
                        }
                    } else {
                        if (placed && in[q])
                            *reinterpret_cast<uint4*>(to + q * LPR * kChunkBytes) = make_uint4(y[q][0], y[q][1], y[q][2], y[q][3]);
                    }
                }
            }
        }
        h3qk::cp_async_wait<0>();
    }
}

// ---------------------------------------------------------------------------
// Reading back: a thread takes 8 channels of kReadRows rows of a head at a
// time, `turns` times, the next turn's rows on their way; K in one half of the
// grid and V in the other.  Small calls spread over the GPU in one turn.  Four
// caches of up to 32,768 keys, 8 K/V heads of 128, 4 bits to bf16: 104 us, 6.1
// TB/s; 157 in one turn a thread.  Bound by HBM: mostly
// the dense rows' 2 bytes a value on their way out.
// ---------------------------------------------------------------------------
constexpr int kReadRows = 3, kReadTurns = 8;

struct ReadArgs {
    Pool c;
    const int32_t* starts;
    int64_t rows;
    int32_t turns;
    uint16_t* out[2];
};

template <bool BF16, bool E2M1>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ ReadArgs a)
{
    const Pool& c = a.c;
    const int item = blockIdx.y / c.kv_heads, head = blockIdx.y % c.kv_heads;
    const bool is_v = blockIdx.z != 0;
    const int chunk = threadIdx.x;
    const int keys = keys_of(c, item), start = a.starts ? max(__ldg(a.starts + item), 0) : 0;
    const int32_t* table = c.table + item * c.table_stride;
    const uint8_t* data = is_v ? c.v + head * c.v_head : c.k + head * c.k_head;
    const uint8_t* scales = is_v ? c.v_scales + head * c.vs_head : c.k_scales + head * c.ks_head;
    const int64_t page_bytes = is_v ? c.v_page : c.k_page, row_bytes = is_v ? c.v_row : c.k_row;
    const int64_t scale_page = is_v ? c.vs_page : c.ks_page;
    const float tensor_scale = is_v ? c.v_scale : c.k_scale;
    const int64_t step = static_cast<int64_t>(blockDim.y) * kReadRows;
    const int64_t end = min(a.rows, (blockIdx.x + int64_t{1}) * step * a.turns);
    uint4 got[kReadRows];
    uint32_t scale[kReadRows];
    auto fetch = [&](int64_t first) {
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
            const int64_t r = first + u * blockDim.y, at = start + r;
            got[u] = make_uint4(0, 0, 0, 0);
            scale[u] = 0;
            if (r >= end || at >= keys) continue;
            const int page = page_of(c, table, static_cast<int>(at));
            if (page < 0) continue;
            const int in_page = static_cast<int>(at) & ((1 << c.page_shift) - 1);
            const uint8_t* from = data + page * page_bytes + in_page * row_bytes;
            if constexpr (E2M1) {
                got[u].x = __ldcs(reinterpret_cast<const uint32_t*>(from) + chunk);
                scale[u] = __ldg(scales + page * scale_page + static_cast<int64_t>(in_page) * (c.dim / 16) + chunk / 2);
            } else {
                got[u] = __ldcs(reinterpret_cast<const uint4*>(from) + chunk);
            }
        }
    };
    int64_t first = blockIdx.x * step * a.turns + threadIdx.y;
    fetch(first);
    for (; first < end; first += step) {
        uint4 now[kReadRows];
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
            now[u] = got[u];
            if constexpr (E2M1) now[u].y = scale[u];
        }
        if (first + step < end) fetch(first + step);  // the next turn's rows are on their way
#pragma unroll
        for (int u = 0; u < kReadRows; ++u) {
            const int64_t r = first + u * blockDim.y;
            if (r >= end) continue;
            if constexpr (E2M1) {
                uint32_t v[4], w[4];
                widen_codes(now[u].x, v);
                const uint32_t g = widen_scales(now[u].y * 0x101u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the product of code and scale is exact
                    const float2 f = h3qk::widen2<false>(mul_half2(v[i], g));
                    w[i] = h3qk::round2<BF16>(__fmul_rn(f.x, tensor_scale), __fmul_rn(f.y, tensor_scale));
                }
                now[u] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __stcs(reinterpret_cast<uint4*>(a.out[is_v ? 1 : 0] + (static_cast<int64_t>(blockIdx.y) * a.rows + r) * c.dim) + chunk,
                   now[u]);
        }
    }
}

// P: chunks of a head row, to a power of two; two of them a lane.
template <bool BF16>
cudaError_t launch_append(int P, bool e2m1, const AppendArgs& a, int blocks, cudaStream_t st)
{
    constexpr int kThreads = 32 * kWarps;
    if (e2m1) {
        switch (P) {
        case 4: append_kernel<BF16, 2, 2, true><<<blocks, kThreads, 0, st>>>(a); break;
        case 8: append_kernel<BF16, 4, 2, true><<<blocks, kThreads, 0, st>>>(a); break;
        default: append_kernel<BF16, 8, 2, true><<<blocks, kThreads, 0, st>>>(a); break;
        }
    } else {
        switch (P) {
        case 1: append_kernel<BF16, 1, 1, false><<<blocks, kThreads, 0, st>>>(a); break;
        case 2: append_kernel<BF16, 1, 2, false><<<blocks, kThreads, 0, st>>>(a); break;
        case 4: append_kernel<BF16, 2, 2, false><<<blocks, kThreads, 0, st>>>(a); break;
        case 8: append_kernel<BF16, 4, 2, false><<<blocks, kThreads, 0, st>>>(a); break;
        default: append_kernel<BF16, 8, 2, false><<<blocks, kThreads, 0, st>>>(a); break;
        }
    }
    h3qk_internal_count_launch();
    return cudaGetLastError();
}

// The bytes of one pool tensor: rows of row_bytes, their steps in bytes.
struct Step {
    int64_t step, n;
};
struct Span {
    int64_t page, head, row, row_bytes;
    int64_t all(const h3qk_cache& c) const  // from its first byte to its last
    {
        return c.pages ? (c.pages - 1) * page + (c.kv_heads - 1) * head + (c.page_size - 1) * row + row_bytes : 0;
    }
    // Its dimensions of more than one entry, the widest step first.
    int steps(const h3qk_cache& c, Step (&d)[3]) const
    {
        const Step from[3] = {{page, c.pages}, {head, c.kv_heads}, {row, c.page_size}};
        int n = 0;
        for (const Step& s : from) {
            if (s.n == 1) continue;
            int at = n++;
            for (; at > 0 && d[at - 1].step < s.step; --at) d[at] = d[at - 1];
            d[at] = s;
        }
        return n;
    }
};

// Strides of one tensor in bytes; those of single-entry dimensions are replaced by ones that fit.
h3qk_status check_strides(const h3qk_cache& c, const void* data, h3qk_strides s, int64_t row_bytes, int64_t size, bool gaps,
                          Span* out)
{
    if (!data && c.pages > 0) return H3QK_ERR_INVALID_ARG;
    const int64_t most = (INT64_C(1) << 36) / size;
    if (c.kv_heads == 1) s.head = c.page_size * s.row;
    if (c.pages <= 1) s.item = c.kv_heads * s.head;
    if (s.row * size < row_bytes || s.head <= 0 || s.item <= 0) return H3QK_ERR_INVALID_ARG;
    if (!gaps && s.row * size != row_bytes) return H3QK_ERR_INVALID_ARG;
    if (s.row >= most || s.head >= most || s.item >= most) return H3QK_ERR_INVALID_ARG;
    out->row = s.row * size;
    out->head = s.head * size;
    out->page = s.item * size;
    out->row_bytes = row_bytes;
    if ((gaps && out->row % 16) || out->head % 16 || out->page % 16 || !aligned(data, 16)) return H3QK_ERR_MISALIGNED;
    const double span = static_cast<double>(c.pages) * out->page + static_cast<double>(c.kv_heads) * out->head +
                        static_cast<double>(c.page_size) * out->row;
    return span > 1e15 ? H3QK_ERR_INVALID_ARG : H3QK_OK;
}

// Rows of a tensor that is written may not run into one another: each
// dimension steps over the ones inside it.
bool disjoint_rows(const Span& s, const h3qk_cache& c)
{
    Step d[3];
    int64_t reach = s.row_bytes;
    for (int i = s.steps(c, d) - 1; i >= 0; --i) {
        if (d[i].step < reach) return false;
        reach += d[i].step * (d[i].n - 1);
    }
    return true;
}

int64_t reach_of(const Step* d, int n, int64_t row_bytes)
{
    for (int i = 0; i < n; ++i) row_bytes += d[i].step * (d[i].n - 1);
    return row_bytes;
}

// Whether two tensors of a pool, the second `apart` bytes behind the first, share
// bytes; each is disjoint in itself.  Where their widest steps are the same,
// what lies inside one may lie between the steps of the other (K and V of a
// page, of a head or of a row beside each other): the few pairs of their blocks
// that could meet are looked at.  Else their whole extents count.
bool collide(const Step* x, int nx, int64_t x_row, const Step* y, int ny, int64_t y_row, int64_t apart)
{
    if (apart >= reach_of(x, nx, x_row) || -apart >= reach_of(y, ny, y_row)) return false;
    if (nx == 0 || ny == 0 || x->step != y->step || x->n != y->n) return true;
    const int64_t step = x->step, in_x = reach_of(x + 1, nx - 1, x_row), in_y = reach_of(y + 1, ny - 1, y_row);
    // block i + t of the second starts apart + t step behind block i of the first
    int64_t first = (-in_y - apart) / step - 1, last = (in_x - apart) / step + 1;
    if (first < 1 - x->n) first = 1 - x->n;
    if (last > x->n - 1) last = x->n - 1;
    for (int64_t t = first; t <= last; ++t)
        if (collide(x + 1, nx - 1, x_row, y + 1, ny - 1, y_row, apart + t * step)) return true;
    return false;
}
bool collide(const void* a, const Span& x, const void* b, const Span& y, const h3qk_cache& c)
{
    if (c.pages == 0) return false;
    Step dx[3], dy[3];
    const int nx = x.steps(c, dx), ny = y.steps(c, dy);
    return collide(dx, nx, x.row_bytes, dy, ny, y.row_bytes,
                   static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)));
}

}  // namespace

h3qk_status h3qk_pages::check_pool(const h3qk_cache* cache, bool written, Pool* pool, PoolRanges* ranges)
{
    if (!cache) return H3QK_ERR_INVALID_ARG;
    const h3qk_cache& c = *cache;
    const bool e2m1 = c.format == H3QK_E2M1;
    if (!e2m1 && c.format != H3QK_FP16 && c.format != H3QK_BF16) return H3QK_ERR_INVALID_ARG;
    if (c.kv_heads < 1 || c.kv_heads > 65535 || c.batch < 1 || c.batch > 65535) return H3QK_ERR_INVALID_ARG;
    const int step = e2m1 ? 32 : 8;
    if (c.head_dim < step || c.head_dim > 128 || c.head_dim % step) return H3QK_ERR_INVALID_ARG;
    if (c.page_size < 16 || c.page_size > 65536 || (c.page_size & (c.page_size - 1))) return H3QK_ERR_INVALID_ARG;
    if (c.pages < 0 || c.pages >= (INT64_C(1) << 31) || c.max_pages < 0) return H3QK_ERR_INVALID_ARG;
    if (static_cast<int64_t>(c.max_pages) * c.page_size >= (INT64_C(1) << 30)) return H3QK_ERR_INVALID_ARG;
    const int64_t stride = c.table_stride ? c.table_stride : c.max_pages;
    if (stride < c.max_pages || stride > (INT64_C(1) << 40)) return H3QK_ERR_INVALID_ARG;
    if (!c.kv_lens || (!c.block_table && c.max_pages > 0)) return H3QK_ERR_INVALID_ARG;
    if (!aligned(c.kv_lens, 4) || !aligned(c.block_table, 4)) return H3QK_ERR_MISALIGNED;
    // Between these every step of the rounding is a normal binary32 number: the smallest
    // group scale times k_scale is 2^-126, and 1 / (6 k_scale) well above that.
    for (const float ts : {c.k_scale, c.v_scale})
        if (ts != 0.0f && !(ts >= 0x1p-117f && ts <= 0x1p117f)) return H3QK_ERR_INVALID_ARG;
    if (!e2m1 && ((c.k_scale != 0.0f && c.k_scale != 1.0f) || (c.v_scale != 0.0f && c.v_scale != 1.0f) || c.k_scales ||
                  c.v_scales))
        return H3QK_ERR_INVALID_ARG;
    Span s[4] = {};
    const int64_t row = e2m1 ? c.head_dim / 2 : c.head_dim * 2;
    h3qk_status st;
    if ((st = check_strides(c, c.k, c.k_strides, row, e2m1 ? 1 : 2, !e2m1, &s[0])) != H3QK_OK) return st;
    if ((st = check_strides(c, c.v, c.v_strides, row, e2m1 ? 1 : 2, !e2m1, &s[1])) != H3QK_OK) return st;
    void* const data[4] = {c.k, c.v, c.k_scales, c.v_scales};
    const int parts = e2m1 ? 4 : 2;
    if (e2m1) {
        if ((st = check_strides(c, c.k_scales, c.k_scale_strides, c.head_dim / 16, 1, false, &s[2])) != H3QK_OK) return st;
        if ((st = check_strides(c, c.v_scales, c.v_scale_strides, c.head_dim / 16, 1, false, &s[3])) != H3QK_OK) return st;
    }
    if (written) {
        for (int i = 0; i < parts; ++i)
            if (!disjoint_rows(s[i], c)) return H3QK_ERR_ALIAS;
        for (int i = 0; i < parts; ++i)
            for (int k = i + 1; k < parts; ++k)
                if (collide(data[i], s[i], data[k], s[k], c)) return H3QK_ERR_ALIAS;
    }
    for (int i = 0; i < 4; ++i) ranges->data[i] = range_of(data[i], i < parts ? s[i].all(c) : 0);
    ranges->lists[0] = range_of(c.block_table, c.max_pages ? ((c.batch - 1) * stride + c.max_pages) * 4 : 0);
    ranges->lists[1] = range_of(c.kv_lens, c.batch * 4);
    Pool& p = *pool;
    p.k = static_cast<uint8_t*>(c.k);
    p.v = static_cast<uint8_t*>(c.v);
    p.k_scales = static_cast<uint8_t*>(c.k_scales);
    p.v_scales = static_cast<uint8_t*>(c.v_scales);
    p.k_page = s[0].page, p.k_head = s[0].head, p.k_row = s[0].row;
    p.v_page = s[1].page, p.v_head = s[1].head, p.v_row = s[1].row;
    p.ks_page = s[2].page, p.ks_head = s[2].head;
    p.vs_page = s[3].page, p.vs_head = s[3].head;
    p.k_page16 = static_cast<uint32_t>(s[0].page / 16), p.v_page16 = static_cast<uint32_t>(s[1].page / 16);
    p.ks_page16 = static_cast<uint32_t>(s[2].page / 16), p.vs_page16 = static_cast<uint32_t>(s[3].page / 16);
    p.table = c.block_table;
    p.table_stride = stride;
    p.kv_lens = c.kv_lens;
    p.pages = static_cast<int32_t>(c.pages);
    p.max_pages = c.max_pages;
    p.batch = c.batch;
    p.kv_heads = c.kv_heads;
    p.dim = c.head_dim;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
    p.k_scale = c.k_scale > 0.0f ? c.k_scale : 1.0f;
    p.v_scale = c.v_scale > 0.0f ? c.v_scale : 1.0f;
    return H3QK_OK;
}

extern "C" h3qk_status h3qk_cache_append(const h3qk_cache* cache, const void* qkv, const float* norm_wq,
                                         const float* norm_wk, const int32_t* positions, int64_t tokens, int32_t heads,
                                         int32_t rotary_dim, const int32_t* q_offsets, void* out_q, const h3qk_opts* opts,
                                         h3qk_stream_t stream)
{
    AppendArgs a = {};
    PoolRanges pool;
    h3qk_status s = check_pool(cache, true, &a.c, &pool);
    if (s != H3QK_OK) return s;
    const bool e2m1 = cache->format == H3QK_E2M1;
    h3qk_opts o;
    h3qk_opts_init(&o);
    if (opts) o = *opts;
    o.batch = 1;
    o.out_layout = H3QK_LAYOUT_HEAD_MAJOR;
    o.valid_lens = nullptr;
    o.sat_counts = nullptr;
    if (heads < 1 || heads > 65535 || heads + 2 * a.c.kv_heads > 65536) return H3QK_ERR_INVALID_ARG;
    if (tokens < 0 || tokens >= (INT64_C(1) << 30)) return H3QK_ERR_INVALID_ARG;
    if (!q_offsets && tokens % a.c.batch) return H3QK_ERR_INVALID_ARG;
    if (!aligned(q_offsets, 4)) return H3QK_ERR_MISALIGNED;
    if (tokens > 0 && rotary_dim > 0 && !positions && o.n_axes != 1) return H3QK_ERR_INVALID_ARG;
    // A packed row is one part of heads + 2 kv_heads head rows.  Without
    // positions the row's place takes their role (the checks see no rows then,
    // and what they would say of the rows follows here).
    const int32_t all = heads + 2 * a.c.kv_heads;
    h3qk_detail::Plan pl;
    const bool given = positions || rotary_dim == 0;
    s = h3qk_detail::plan_inputs(qkv, norm_wq, norm_wk, positions, given ? tokens : 0, all, a.c.dim, rotary_dim, 0,
                                 e2m1 ? H3QK_BF16 : cache->format, o, stream, &pl, 1);
    if (s != H3QK_OK) return s;
    if (!e2m1 && pl.bf16 != (cache->format == H3QK_BF16)) return H3QK_ERR_INVALID_ARG;
    if (!given) {
        if (tokens > 0 && (!qkv || pl.p.row_stride > (INT64_C(1) << 40) / tokens)) return H3QK_ERR_INVALID_ARG;
        pl.p.rows = tokens;
        pl.ins[0] = range_of(qkv, tokens > 0 ? ((tokens - 1) * pl.p.row_stride + pl.HD) * 2 : 0);
    }
    if (tokens > 0 && !out_q) return H3QK_ERR_INVALID_ARG;
    if (!aligned(out_q, 16)) return H3QK_ERR_MISALIGNED;
    const Range out = range_of(out_q, tokens * heads * a.c.dim * 2);
    const Range offsets = range_of(q_offsets, q_offsets ? (a.c.batch + 1) * 4 : 0);
    const Range outs[5] = {out, pool.data[0], pool.data[1], pool.data[2], pool.data[3]};
    for (int i = 0; i < 5; ++i) {
        if (i > 0 && overlap(out, outs[i])) return H3QK_ERR_ALIAS;
        if (overlap(outs[i], offsets) || overlap(outs[i], pool.lists[0]) || overlap(outs[i], pool.lists[1]))
            return H3QK_ERR_ALIAS;
        if (h3qk_detail::overlaps_inputs(pl, outs[i])) return H3QK_ERR_ALIAS;
    }
    if (tokens == 0) return H3QK_OK;
    a.p = pl.p;
    a.offsets = q_offsets;
    a.each = q_offsets ? 0 : static_cast<int32_t>(tokens / a.c.batch);
    a.q_heads = heads;
    a.out_q = static_cast<uint16_t*>(out_q);
    a.to_scale[0] = static_cast<float>(1.0 / (6.0 * a.c.k_scale));
    a.to_scale[1] = static_cast<float>(1.0 / (6.0 * a.c.v_scale));
    const int tpw = pl.P == 1 ? 32 : 64 / pl.P;
    a.groups = (tokens + tpw - 1) / tpw;
    // Heads are cut into slices so that a warp's turns, at the cost of a
    // slice's heads and about eight heads' worth of search and angles each,
    // are fewest: one token's heads spread over the GPU, many rows' do not.
    const int cap = kBlocks * h3qk_internal_sm_count();
    const int64_t warps = static_cast<int64_t>(cap) * kWarps;
    int64_t least = INT64_MAX;
    for (int32_t slices = 1; slices <= (all + 3) / 4; ++slices) {
        const int32_t h = ((all + slices - 1) / slices + 3) / 4 * 4;
        const int64_t n = (all + h - 1) / h;
        const int64_t cost = (a.groups * n + warps - 1) / warps * (h + 8);
        if (cost < least) {
            least = cost;
            a.slice_heads = h;
            a.slices = static_cast<int32_t>(n);
        }
    }
    const int64_t want = (a.groups * a.slices + kWarps - 1) / kWarps;
    const int blocks = static_cast<int>(want < cap ? want : cap);
    return status_of(pl.bf16 ? launch_append<true>(pl.P, e2m1, a, blocks, pl.st)
                             : launch_append<false>(pl.P, e2m1, a, blocks, pl.st));
}

extern "C" h3qk_status h3qk_cache_read(const h3qk_cache* cache, const int32_t* starts, int64_t rows, h3qk_dtype dtype,
                                       void* out_k, void* out_v, h3qk_stream_t stream)
{
    ReadArgs a = {};
    PoolRanges pool;
    const h3qk_status s = check_pool(cache, false, &a.c, &pool);
    if (s != H3QK_OK) return s;
    if (dtype != H3QK_FP16 && dtype != H3QK_BF16) return H3QK_ERR_INVALID_ARG;
    const bool e2m1 = cache->format == H3QK_E2M1;
    if (!e2m1 && cache->format != dtype) return H3QK_ERR_INVALID_ARG;
    if (rows < 0 || rows >= (INT64_C(1) << 30)) return H3QK_ERR_INVALID_ARG;
    if (!aligned(starts, 4)) return H3QK_ERR_MISALIGNED;
    const int64_t slots = static_cast<int64_t>(a.c.batch) * a.c.kv_heads;
    if (slots > 65535) return H3QK_ERR_INVALID_ARG;
    const int64_t bytes = slots * rows * a.c.dim * 2;
    if (bytes > 0 && (!out_k || !out_v)) return H3QK_ERR_INVALID_ARG;
    if (!aligned(out_k, 16) || !aligned(out_v, 16)) return H3QK_ERR_MISALIGNED;
    const Range outs[2] = {range_of(out_k, bytes), range_of(out_v, bytes)};
    if (overlap(outs[0], outs[1])) return H3QK_ERR_ALIAS;
    for (const Range& o : outs) {
        for (const Range& d : pool.data)
            if (overlap(o, d)) return H3QK_ERR_ALIAS;
        if (overlap(o, pool.lists[0]) || overlap(o, pool.lists[1]) || overlap(o, range_of(starts, starts ? a.c.batch * 4 : 0)))
            return H3QK_ERR_ALIAS;
    }
    if (bytes == 0) return H3QK_OK;
    a.starts = starts;
    a.rows = rows;
    a.out[0] = static_cast<uint16_t*>(out_k);
    a.out[1] = static_cast<uint16_t*>(out_v);
    const int chunks = a.c.dim / 8, per = 256 / chunks;
    const dim3 block(chunks, per);
    const int64_t one_turn = (rows + per * kReadRows - 1) / (per * kReadRows);
    const int64_t turns = one_turn * slots * 2 / (8 * h3qk_internal_sm_count());
    a.turns = static_cast<int32_t>(turns < 1 ? 1 : turns > kReadTurns ? kReadTurns : turns);
    const int64_t a_block = static_cast<int64_t>(per) * kReadRows * a.turns;
    const dim3 grid(static_cast<unsigned>((rows + a_block - 1) / a_block), static_cast<unsigned>(slots), 2);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == H3QK_BF16;
    if (e2m1) {
        if (bf16) read_kernel<true, true><<<grid, block, 0, st>>>(a);
        else read_kernel<false, true><<<grid, block, 0, st>>>(a);
    } else {
        if (bf16) read_kernel<true, false><<<grid, block, 0, st>>>(a);
        else read_kernel<false, false><<<grid, block, 0, st>>>(a);
    }
    h3qk_internal_count_launch();
    return status_of(cudaGetLastError());
}
