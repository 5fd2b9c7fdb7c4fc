// Host side of attention: argument checks, tensor maps and the choice of
// kernels.
#include <cudaTypedefs.h>

#include <cmath>

#include "h3qk_attn.cuh"

namespace {

using h3qk_core::Maps;
using h3qk_core::Params;
using h3qk_core::Strides;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

static __device__ unsigned int g_stuck;

struct Tensor {
    const void* data;
    h3qk_strides s;
    int64_t heads, rows;
};

// A tensor's strides, with those of single-entry dimensions replaced by ones
// that fit; false when one is out of range.
h3qk_status check_tensor(Tensor& t, int64_t batch, int64_t dim, Range* r)
{
    if (batch * t.heads * t.rows == 0) {
        *r = range_of(t.data, 0);
        return H3QK_OK;
    }
    if (!t.data) return H3QK_ERR_INVALID_ARG;
    if (t.rows == 1) t.s.row = dim;
    if (t.heads == 1) t.s.head = t.s.row;
    if (batch == 1) t.s.item = t.s.row;
    const int64_t most = INT64_C(1) << 38;  // the tensor maps' strides stay below 2^40 bytes
    if (t.s.row < dim || t.s.head <= 0 || t.s.item <= 0) return H3QK_ERR_INVALID_ARG;
    if (t.s.row >= most || t.s.head >= most || t.s.item >= most) return H3QK_ERR_INVALID_ARG;
    if (t.s.row % 8 || t.s.head % 8 || t.s.item % 8 || !aligned(t.data, 16)) return H3QK_ERR_MISALIGNED;
    const double span = static_cast<double>(t.rows - 1) * t.s.row + static_cast<double>(t.heads - 1) * t.s.head +
                        static_cast<double>(batch - 1) * t.s.item;
    if (span > 1e15) return H3QK_ERR_INVALID_ARG;
    *r = range_of(t.data, ((t.rows - 1) * t.s.row + (t.heads - 1) * t.s.head + (batch - 1) * t.s.item + dim) * 2);
    return H3QK_OK;
}

Strides plain(const h3qk_strides& s) { return Strides{s.item, s.head, s.row}; }

// Rows of an output whose dimensions interleave may not run into one another:
// ordered by stride, each dimension must step over the one before it.
bool disjoint_rows(const Tensor& t, int64_t batch, int64_t dim)
{
    int64_t step[3] = {t.s.row, t.s.head, t.s.item}, n[3] = {t.rows, t.heads, batch};
    for (int i = 0; i < 2; ++i)
        for (int k = 0; k < 2 - i; ++k)
            if (step[k] > step[k + 1]) {
                std::swap(step[k], step[k + 1]);
                std::swap(n[k], n[k + 1]);
            }
    int64_t reach = dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (step[i] < reach) return false;
        reach += step[i] * (n[i] - 1);
    }
    return true;
}

// Few rows: tiles of 16 that all heads of a K/V head share, against tiles of
// 256 of each head.  The first read the cache once a tile of 16, the second
// once a head and at the tensor cores' rate, so the first serve while they
// are fewer than about two thirds of the heads.  Measured, 40 heads on 8 of
// 128, 8 x 8,192 keys: 1 / 2 / 3 / 5 tiles of 16 take 62 / 110 / 161 / 247 us,
// tiles of 256 take 177; 16 heads on 16 of 64, 4,896 keys: 1 / 2 take 12.1 /
// 16.9 us against 11.8.
int64_t row_tiles(const h3qk_attn& a) { return (a.q_rows * (a.heads / a.kv_heads) + 15) / 16; }

bool use_split(const h3qk_attn& a)
{
    const int64_t most = 2 * (a.heads / a.kv_heads) / 3;
    return a.docs == 0 && row_tiles(a) <= (most > 1 ? most : 1);
}

// How the split kernel cuts the keys: into one block for each that the SMs
// hold at once (4 an SM up to 64 channels, 2 beyond: their shared memory), over
// the whole call, but into chunks of at least 128 keys (two turns of a block's
// four warps) and at most 2,048 (uneven caches still fill the SMs).
void split_of(const h3qk_attn& a, int32_t* splits, int32_t* chunk)
{
    const int64_t base = static_cast<int64_t>(a.batch) * a.kv_heads * row_tiles(a);
    const int64_t slots = (a.head_dim <= 64 ? 4 : 2) * static_cast<int64_t>(h3qk_internal_sm_count());
    const int64_t want = base < slots ? slots / base : 1;
    int64_t c = (a.kv_rows + want - 1) / want;
    c = (c + 63) / 64 * 64;
    c = c < 128 ? 128 : c > 2048 ? 2048 : c;
    if (a.kv_rows <= 256) c = 256;  // one chunk and no second kernel
    // the grid's first dimension and the join's loop stay small
    while ((a.kv_rows + c - 1) / c > 4096) c *= 2;
    *chunk = static_cast<int32_t>(c);
    *splits = static_cast<int32_t>(a.kv_rows > 0 ? (a.kv_rows + c - 1) / c : 1);
}

// The tail is worth a second kernel (about 5 us) where it saves some eight key
// tiles of 128 (about 1 us each) of the last round; a part keeps at least
// four.  16 heads of 4896 x 64 are 2.1 rounds of tiles: 118 us whole, 104 cut;
// 10 heads of 4096 x 128, 1.05 rounds: 106 and 75; 2 heads of 2000 x 64: 23
// and 16.  Row lengths and documents on the device leave tiles empty: after a
// first full round nothing is known of the last one then, and it stays whole
// (16 heads whose lengths made two rounds exactly: 89 us whole, 102 cut).
// Causal tiles go longest first, so that after a full round the last ones are
// the shortest and fill up behind the others: whole, 16 heads of 4896 x 64
// take 59 us (cut 66), 10 of 4096 x 128 51 (55), 40 on 8 of 8160 x 128 420
// (431).  A prefix makes all tiles as long as it is, which only the device
// knows: with a quarter of the rows 67 us whole and 69 cut, with all of them
// 119 and 104, so there the tail is cut.
h3qk_core::TilePlan tile_plan(const h3qk_attn& a)
{
    constexpr int64_t kRows = h3qk_core::kRowTile;
    h3qk_core::TilePlan t;
    t.tiles = (a.q_rows + kRows - 1) / kRows + a.docs;
    const int64_t total = t.tiles * a.heads * a.batch, sms = h3qk_internal_sm_count();
    t.tail = total % sms;
    t.parts = 1;
    const bool short_tail = a.causal && !a.prefix_lens;
    if (t.tail > 0 && (total < sms || !(a.q_lens || a.docs || short_tail))) {
        const int64_t keys = (a.kv_rows + 127) / 128;
        t.parts = sms / t.tail;
        if (t.parts > keys / 4) t.parts = keys / 4;
        if (t.parts > 16) t.parts = 16;
        if (t.parts < 2 || keys - keys / t.parts < 8) t.parts = 1;
    }
    if (t.parts == 1) t.tail = 0;
    t.whole = total - t.tail;
    return t;
}

h3qk_status check_sizes(const h3qk_attn& a)
{
    if (a.dtype != H3QK_FP16 && a.dtype != H3QK_BF16) return H3QK_ERR_INVALID_ARG;
    if (a.batch < 1 || a.batch > 65535 || a.heads < 1 || a.heads > 65535) return H3QK_ERR_INVALID_ARG;
    if (a.kv_heads < 1 || a.heads % a.kv_heads) return H3QK_ERR_INVALID_ARG;
    if (a.head_dim < 8 || a.head_dim > 128 || a.head_dim % 8) return H3QK_ERR_INVALID_ARG;
    const int64_t most = INT64_C(1) << 30;
    if (a.q_rows < 0 || a.kv_rows < 0 || a.q_rows >= most || a.kv_rows >= most) return H3QK_ERR_INVALID_ARG;
    if (a.causal != 0 && a.causal != 1) return H3QK_ERR_INVALID_ARG;
    if (!(a.scale >= 0.0f) || !std::isfinite(a.scale)) return H3QK_ERR_INVALID_ARG;
    if (!(a.softcap >= 0.0f) || !std::isfinite(a.softcap)) return H3QK_ERR_INVALID_ARG;
    if (a.reserved != 0 || a.docs < 0 || a.docs > (1 << 20)) return H3QK_ERR_INVALID_ARG;
    if (a.docs > 0 && (a.batch != 1 || a.q_rows != a.kv_rows || !a.doc_offsets || a.q_lens || a.kv_lens || a.q_starts))
        return H3QK_ERR_INVALID_ARG;
    if (a.docs == 0 && a.doc_offsets) return H3QK_ERR_INVALID_ARG;
    if (a.prefix_lens && !a.causal) return H3QK_ERR_INVALID_ARG;
    return H3QK_OK;
}

h3qk_status check_lists(const h3qk_attn& a, Range (&lists)[6])
{
    const int32_t* i32[5] = {a.prefix_lens, a.doc_offsets, a.q_lens, a.kv_lens, a.q_starts};
    const int64_t n[5] = {a.docs ? a.docs : a.batch, a.docs + 1, a.batch, a.batch, a.batch};
    if (!aligned(a.slopes, 4)) return H3QK_ERR_MISALIGNED;
    lists[5] = range_of(a.slopes, a.slopes ? a.heads * 4 : 0);
    for (int k = 0; k < 5; ++k) {
        if (!aligned(i32[k], 4)) return H3QK_ERR_MISALIGNED;
        lists[k] = range_of(i32[k], i32[k] ? n[k] * 4 : 0);
    }
    return H3QK_OK;
}

using Encode = PFN_cuTensorMapEncodeTiled_v12000;

// The driver's tensor-map encoder (looked up once; a race finds the same address).
Encode encoder()
{
    static Encode fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<Encode>(p);
    }
    return fn;
}

bool encode(CUtensorMap* m, const Tensor& t, bool bf16, int64_t batch, int64_t dim)
{
    return h3qk_core::encode_map(m, t.data, bf16, dim, t.rows, t.heads, batch, t.s.row * 2, t.s.head * 2, t.s.item * 2, 128);
}

using h3qk_core::no_maps;
using h3qk_core::stuck_addr;
void fill(Params& p, const h3qk_attn& a)
{
    p.batch = a.batch;
    p.heads = a.heads;
    p.kv_heads = a.kv_heads;
    p.group = a.heads / a.kv_heads;
    p.dim = a.head_dim;
    p.q_rows = static_cast<int32_t>(a.q_rows);
    p.kv_rows = static_cast<int32_t>(a.kv_rows);
    p.causal = a.causal;
    p.docs = a.docs;
    p.scale = a.scale > 0.0f ? a.scale : 1.0f / std::sqrt(static_cast<float>(a.head_dim));
    p.cap = a.softcap;
    p.slopes = a.slopes;
    p.prefix_lens = a.prefix_lens;
    p.doc_offsets = a.doc_offsets;
    p.q_lens = a.q_lens;
    p.kv_lens = a.kv_lens;
    p.q_starts = a.q_starts;
    p.lse = a.lse;
}

}  // namespace

bool h3qk_core::encode_map(CUtensorMap* m, const void* data, bool bf16, int64_t dim, int64_t rows, int64_t heads, int64_t items,
                           int64_t row_bytes, int64_t head_bytes, int64_t item_bytes, int box_rows)
{
    const Encode fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(items)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(head_bytes),
                                   static_cast<cuuint64_t>(item_bytes)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1}, ones[4] = {1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(data), dims,
              strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

unsigned int* h3qk_core::stuck_addr()
{
    static unsigned int* addr[64] = {nullptr};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    if (!addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_stuck) != cudaSuccess) return nullptr;
        addr[dev] = static_cast<unsigned int*>(p);
    }
    return addr[dev];
}

// The runtime could not give the stuck counter or a tensor map.
h3qk_status h3qk_core::no_maps()
{
    const cudaError_t e = cudaGetLastError();
    return h3qk_internal_fail_cuda(e != cudaSuccess ? e : cudaErrorInvalidValue);
}

extern "C" size_t h3qk_attention_workspace_bytes(const h3qk_attn* call)
{
    if (!call || check_sizes(*call) != H3QK_OK) return 0;
    const h3qk_attn& a = *call;
    if (!use_split(a)) {
        const h3qk_core::TilePlan t = tile_plan(a);
        return static_cast<size_t>(t.tail * t.parts) * h3qk_core::tile_part_floats(a.head_dim) * 4;
    }
    int32_t splits, chunk;
    split_of(a, &splits, &chunk);
    if (splits == 1) return 0;
    return static_cast<size_t>(a.batch) * a.kv_heads * row_tiles(a) * splits * 16 * (a.head_dim + 2) * 4;
}

extern "C" h3qk_status h3qk_attention(const h3qk_attn* call, h3qk_stream_t stream)
{
    if (!call) return H3QK_ERR_INVALID_ARG;
    const h3qk_attn& a = *call;
    h3qk_status s = check_sizes(a);
    if (s != H3QK_OK) return s;
    Tensor t[4] = {{a.q, a.q_strides, a.heads, a.q_rows},
                   {a.k, a.k_strides, a.kv_heads, a.kv_rows},
                   {a.v, a.v_strides, a.kv_heads, a.kv_rows},
                   {a.out, a.out_strides, a.heads, a.q_rows}};
    Range r[4], lists[6];
    for (int i = 0; i < 4; ++i)
        if ((s = check_tensor(t[i], a.batch, a.head_dim, &r[i])) != H3QK_OK) return s;
    if ((s = check_lists(a, lists)) != H3QK_OK) return s;
    if (a.q_rows == 0) return H3QK_OK;
    if (!a.lse) return H3QK_ERR_INVALID_ARG;
    if (!aligned(a.lse, 4)) return H3QK_ERR_MISALIGNED;
    if (!disjoint_rows(t[3], a.batch, a.head_dim)) return H3QK_ERR_ALIAS;
    const size_t need = h3qk_attention_workspace_bytes(call);
    if (need && (!a.workspace || a.workspace_bytes < need)) return H3QK_ERR_INVALID_ARG;
    if (need && !aligned(a.workspace, 16)) return H3QK_ERR_MISALIGNED;
    const Range outs[3] = {r[3], range_of(a.lse, static_cast<int64_t>(a.batch) * a.heads * a.q_rows * 4),
                           range_of(a.workspace, need)};
    for (int i = 0; i < 3; ++i) {
        for (int k = i + 1; k < 3; ++k)
            if (overlap(outs[i], outs[k])) return H3QK_ERR_ALIAS;
        for (int k = 0; k < 3; ++k)
            if (overlap(outs[i], r[k])) return H3QK_ERR_ALIAS;
        for (const Range& l : lists)
            if (overlap(outs[i], l)) return H3QK_ERR_ALIAS;
    }
    Params p = {};
    fill(p, a);
    p.out = static_cast<uint16_t*>(a.out);
    p.os = plain(t[3].s);
    const bool bf16 = a.dtype == H3QK_BF16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (use_split(a)) {
        p.q = static_cast<const uint16_t*>(a.q);
        p.k = static_cast<const uint16_t*>(a.k);
        p.v = static_cast<const uint16_t*>(a.v);
        p.qs = plain(t[0].s);
        p.ks = plain(t[1].s);
        p.vs = plain(t[2].s);
        p.part = static_cast<float*>(a.workspace);
        split_of(a, &p.splits, &p.chunk);
        return h3qk_ops::status_of(h3qk_core::forward_split(bf16, p, st));
    }
    const h3qk_core::TilePlan plan = tile_plan(a);
    if (plan.whole + plan.tail * plan.parts > INT32_MAX) return H3QK_ERR_INVALID_ARG;
    p.tiles = static_cast<int32_t>(plan.tiles);
    p.whole = static_cast<int32_t>(plan.whole);
    p.tail = static_cast<int32_t>(plan.tail);
    p.parts = static_cast<int32_t>(plan.parts);
    p.part = static_cast<float*>(a.workspace);
    Maps m;
    // Without keys no tile is loaded; the maps then describe q instead.
    for (int i = 1; i < 3; ++i)
        if (a.kv_rows == 0) t[i] = t[0];
    p.stuck = stuck_addr();
    if (!p.stuck || !encode(&m.q, t[0], bf16, a.batch, a.head_dim) || !encode(&m.k, t[1], bf16, a.batch, a.head_dim) ||
        !encode(&m.v, t[2], bf16, a.batch, a.head_dim))
        return no_maps();
    return h3qk_ops::status_of(h3qk_core::forward_tiles(bf16, p, m, st));
}

extern "C" size_t h3qk_attention_backward_workspace_bytes(const h3qk_attn* call)
{
    if (!call || check_sizes(*call) != H3QK_OK) return 0;
    return (static_cast<size_t>(call->batch) * call->heads * call->q_rows * 4 + 15) / 16 * 16;
}

extern "C" h3qk_status h3qk_attention_backward(const h3qk_attn* call, h3qk_stream_t stream)
{
    if (!call) return H3QK_ERR_INVALID_ARG;
    const h3qk_attn& a = *call;
    h3qk_status s = check_sizes(a);
    if (s != H3QK_OK) return s;
    constexpr int kIn = 5, kAll = 8;
    Tensor t[kAll] = {{a.q, a.q_strides, a.heads, a.q_rows},
                      {a.k, a.k_strides, a.kv_heads, a.kv_rows},
                      {a.v, a.v_strides, a.kv_heads, a.kv_rows},
                      {a.out, a.out_strides, a.heads, a.q_rows},
                      {a.grad_out, a.grad_out_strides, a.heads, a.q_rows},
                      {a.grad_q, a.grad_q_strides, a.heads, a.q_rows},
                      {a.grad_k, a.grad_k_strides, a.kv_heads, a.kv_rows},
                      {a.grad_v, a.grad_v_strides, a.kv_heads, a.kv_rows}};
    Range r[kAll], lists[6];
    for (int i = 0; i < kAll; ++i)
        if ((s = check_tensor(t[i], a.batch, a.head_dim, &r[i])) != H3QK_OK) return s;
    if ((s = check_lists(a, lists)) != H3QK_OK) return s;
    if (a.q_rows == 0 && a.kv_rows == 0) return H3QK_OK;
    const size_t need = h3qk_attention_backward_workspace_bytes(call);
    if (a.q_rows > 0 && (!a.lse || !a.workspace || a.workspace_bytes < need)) return H3QK_ERR_INVALID_ARG;
    if (!aligned(a.lse, 4) || (need && !aligned(a.workspace, 16))) return H3QK_ERR_MISALIGNED;
    const Range lse = range_of(a.lse, static_cast<int64_t>(a.batch) * a.heads * a.q_rows * 4);
    const Range outs[4] = {r[5], r[6], r[7], range_of(a.workspace, need)};
    for (int i = 0; i < 4; ++i) {
        if (i < 3 && !disjoint_rows(t[kIn + i], a.batch, a.head_dim)) return H3QK_ERR_ALIAS;
        for (int k = i + 1; k < 4; ++k)
            if (overlap(outs[i], outs[k])) return H3QK_ERR_ALIAS;
        for (int k = 0; k < kIn; ++k)
            if (overlap(outs[i], r[k])) return H3QK_ERR_ALIAS;
        for (const Range& l : lists)
            if (overlap(outs[i], l)) return H3QK_ERR_ALIAS;
        if (overlap(outs[i], lse)) return H3QK_ERR_ALIAS;
    }
    Params p = {};
    fill(p, a);
    p.out = static_cast<uint16_t*>(a.out);
    p.os = plain(t[3].s);
    p.dout = static_cast<const uint16_t*>(a.grad_out);
    p.dos = plain(t[4].s);
    p.dq = static_cast<uint16_t*>(a.grad_q);
    p.dqs = plain(t[5].s);
    p.dk = static_cast<uint16_t*>(a.grad_k);
    p.dks = plain(t[6].s);
    p.dv = static_cast<uint16_t*>(a.grad_v);
    p.dvs = plain(t[7].s);
    p.delta = static_cast<float*>(a.workspace);
    p.stuck = stuck_addr();
    // Without rows or without keys nothing is loaded; the maps then describe the other tensors.
    const int of[4] = {a.q_rows ? 0 : 1, a.kv_rows ? 1 : 0, a.kv_rows ? 2 : 0, a.q_rows ? 4 : 1};
    const bool bf16 = a.dtype == H3QK_BF16;
    Maps m;
    CUtensorMap* maps[4] = {&m.q, &m.k, &m.v, &m.dout};
    bool ok = p.stuck != nullptr;
    for (int i = 0; i < 4; ++i) ok = ok && encode(maps[i], t[of[i]], bf16, a.batch, a.head_dim);
    if (!ok) return no_maps();
    return h3qk_ops::status_of(h3qk_core::backward_tiles(bf16, p, m, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" int64_t h3qk_attention_stuck(void)
{
    unsigned int n = 0;
    unsigned int* a = stuck_addr();
    if (!a || cudaMemcpy(&n, a, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return -1;
    return n;
}
