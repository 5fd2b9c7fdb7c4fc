// Layer norm and its gradient.
//   mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both directions are bound by HBM: each element is loaded once, held in
// registers (16-bit elements packed) through both reductions, and written
// once.  A row of up to 32 lanes' worth of elements belongs to one warp
// (eight rows a block, shuffles only); a longer one to a block of its own.
// The variance is the sum of squared deviations from the mean just found,
// not E[x^2] - mean^2, which loses all digits where |mean| >> deviation.
//
// The weight gradient is a sum over all rows.  A block walks its rows with
// every thread on fixed columns, so dw and db grow in registers; each block
// then writes one partial row and a second, chained kernel adds the partial
// rows in a fixed order: no atomics, the same bits on every run.
#include "h3qk_ops.cuh"

namespace {

using namespace h3qk_ops;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

constexpr int kMaxWidth = 16384;  // 512 threads of 32 elements
constexpr int kRowsPerBlock = 8;  // warp-per-row blocks

// VEC neighbouring elements as stored, and as binary32.
template <typename T, int VEC>
struct Pack {
    typename T::raw v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_pack(const typename T::raw* p)
{
    constexpr int bytes = sizeof(typename T::raw) * VEC;
    Pack<T, VEC> r;
    if constexpr (bytes == 16) {
        *reinterpret_cast<uint4*>(r.v) = __ldg(reinterpret_cast<const uint4*>(p));
    } else if constexpr (bytes == 8) {
        *reinterpret_cast<uint2*>(r.v) = __ldg(reinterpret_cast<const uint2*>(p));
    } else if constexpr (bytes == 4) {
        *reinterpret_cast<uint32_t*>(r.v) = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
        r.v[0] = __ldg(p);
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(typename T::raw* p, const Pack<T, VEC>& r)
{
    constexpr int bytes = sizeof(typename T::raw) * VEC;
    if constexpr (bytes == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
    else if constexpr (bytes == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r.v);
    else if constexpr (bytes == 4) *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(r.v);
    else p[0] = r.v[0];
}

template <typename T>
__device__ __forceinline__ float widen(typename T::raw v)
{
    if constexpr (sizeof(v) == 4) return v;
    else if constexpr (T::kBf16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return __half2float(__ushort_as_half(v));
}

template <typename T>
__device__ __forceinline__ typename T::raw narrow(float v)
{
    if constexpr (sizeof(typename T::raw) == 4) return v;
    else if constexpr (T::kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else return __half_as_ushort(__float2half_rn(v));
}

template <int VEC>
__device__ __forceinline__ void load_f32(float (&o)[VEC], const float* p)
{
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
            o[4 * i] = f.x; o[4 * i + 1] = f.y; o[4 * i + 2] = f.z; o[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = __ldg(p + i);
    }
}

struct LnArgs {
    const void* x;
    const void* dy;
    const float* weight;  // [groups, width] or null
    const float* bias;    // the same, or null
    float* stats;         // [rows, 2]: mean, rstd
    void* out;            // y, or dx
    float* partial;       // [groups][parts][2][width]
    int64_t rows_per_group;
    int64_t x_stride, dy_stride, out_stride;
    int32_t width;
    int32_t parts;        // blocks along a group's rows
    float eps, inv_width;
};

// The sum of v over the threads of one row; `slot` alternates so that one
// barrier per sum is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* red, int slot)
{
    v = warp_sum(v);
    if constexpr (!WARP) {
        const int warps = blockDim.x >> 5;
        float* r = red + 32 * slot;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        v = warp_sum(lane < warps ? r[lane] : 0.0f);
    }
    return v;
}

template <typename T, int VEC, int CPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowsPerBlock : 512) layer_norm_kernel(const LnArgs a)
{
    __shared__ float red[64];
    const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int sub = WARP ? (threadIdx.x >> 5) : 0;
    constexpr int kRows = WARP ? kRowsPerBlock : 1;
    const int64_t g = blockIdx.y;
    const float* w = a.weight ? a.weight + g * a.width : nullptr;
    const float* b = a.bias ? a.bias + g * a.width : nullptr;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + sub; r < a.rows_per_group;
         r += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t row = g * a.rows_per_group + r;
        const typename T::raw* x = static_cast<const typename T::raw*>(a.x) + row * a.x_stride;
        Pack<T, VEC> xv[CPT];
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width) xv[k] = load_pack<T, VEC>(x + c);
        }
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s += widen<T>(xv[k].v[i]);
        }
        const float mean = row_sum<WARP>(s, red, 0) * a.inv_width;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = widen<T>(xv[k].v[i]) - mean;
                    s = fmaf(d, d, s);
                }
        }
        const float var = row_sum<WARP>(s, red, 1) * a.inv_width;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (lane == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
        typename T::raw* y = static_cast<typename T::raw*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width) {
                float wv[VEC], bv[VEC];
                if (w) load_f32<VEC>(wv, w + c);
                if (b) load_f32<VEC>(bv, b + c);
                Pack<T, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float v = (widen<T>(xv[k].v[i]) - mean) * rstd;
                    if (w) v *= wv[i];
                    if (b) v += bv[i];
                    o.v[i] = narrow<T>(v);
                }
                store_pack<T, VEC>(y + c, o);
            }
        }
    }
}

template <typename T, int VEC, int CPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowsPerBlock : 512) layer_norm_backward_kernel(const LnArgs a)
{
    extern __shared__ float merge[];  // WARP: [kRowsPerBlock][width], one of dw / db at a time
    __shared__ float red[128];
    allow_dependents();
    const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int lanes = WARP ? 32 : blockDim.x;
    const int sub = WARP ? (threadIdx.x >> 5) : 0;
    constexpr int kRows = WARP ? kRowsPerBlock : 1;
    const int64_t g = blockIdx.y;
    const float* w = a.weight ? a.weight + g * a.width : nullptr;
    float dw[CPT][VEC], db[CPT][VEC];
#pragma unroll
    for (int k = 0; k < CPT; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[k][i] = db[k][i] = 0.0f;

    int slot = 0;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + sub; r < a.rows_per_group;
         r += static_cast<int64_t>(gridDim.x) * kRows, slot ^= 2) {
        const int64_t row = g * a.rows_per_group + r;
        const typename T::raw* x = static_cast<const typename T::raw*>(a.x) + row * a.x_stride;
        const typename T::raw* dy = static_cast<const typename T::raw*>(a.dy) + row * a.dy_stride;
        Pack<T, VEC> xv[CPT], dv[CPT];
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width) {
                xv[k] = load_pack<T, VEC>(x + c);
                dv[k] = load_pack<T, VEC>(dy + c);
            }
        }
        const float2 st = __ldg(reinterpret_cast<const float2*>(a.stats + 2 * row));
        float sg = 0.0f, sgx = 0.0f;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width) {
                float wv[VEC];
                if (w) load_f32<VEC>(wv, w + c);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = widen<T>(dv[k].v[i]);
                    const float xh = (widen<T>(xv[k].v[i]) - st.x) * st.y;
                    const float gi = w ? d * wv[i] : d;
                    sg += gi;
                    sgx = fmaf(gi, xh, sgx);
                    dw[k][i] = fmaf(d, xh, dw[k][i]);
                    db[k][i] += d;
                }
            }
        }
        const float mg = row_sum<WARP>(sg, red, slot) * a.inv_width;
        const float mgx = row_sum<WARP>(sgx, red, slot + 1) * a.inv_width;
        typename T::raw* dx = static_cast<typename T::raw*>(a.out) + row * a.out_stride;
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            const int c = (k * lanes + lane) * VEC;
            if (c < a.width) {
                float wv[VEC];
                if (w) load_f32<VEC>(wv, w + c);
                Pack<T, VEC> o;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = widen<T>(dv[k].v[i]);
                    const float xh = (widen<T>(xv[k].v[i]) - st.x) * st.y;
                    const float gi = w ? d * wv[i] : d;
                    o.v[i] = narrow<T>(st.y * (gi - mg - xh * mgx));
                }
                store_pack<T, VEC>(dx + c, o);
            }
        }
    }
    if (!a.partial) return;
    float* part = a.partial + (g * a.parts + blockIdx.x) * 2 * a.width;
    if constexpr (WARP) {
        // The block's eight warps hold sums of the same columns.
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < CPT; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int c = (k * lanes + lane) * VEC + i;
                    if (c < a.width) merge[sub * a.width + c] = which ? db[k][i] : dw[k][i];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kRowsPerBlock; ++q) s += merge[q * a.width + c];
                part[which * a.width + c] = s;
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int c = (k * lanes + lane) * VEC + i;
                if (c < a.width) {
                    part[c] = dw[k][i];
                    part[a.width + c] = db[k][i];
                }
            }
    }
}

// grad[g][c] = sum over parts of partial[g][part][which][c], parts in order:
// 32 columns a block, 8 lanes of parts, then the 8 sums.
constexpr int kSumCols = 32, kSumLanes = 8;
__global__ void sum_parts_kernel(const float* partial, float* grad_weight, float* grad_bias, int parts, int width)
{
    __shared__ float s[kSumLanes][kSumCols];
    wait_for_previous();
    const int c = blockIdx.x * kSumCols + threadIdx.x;
    const int64_t g = blockIdx.y;
    const int which = blockIdx.z;
    float* grad = which ? grad_bias : grad_weight;
    float v = 0.0f;
    if (c < width)
        for (int p = threadIdx.y; p < parts; p += kSumLanes) v += partial[((g * parts + p) * 2 + which) * width + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < width && grad) {
        v = 0.0f;
#pragma unroll
        for (int q = 0; q < kSumLanes; ++q) v += s[q][threadIdx.x];
        grad[g * width + c] = v;
    }
}

// How a row is spread: elements per load, loads per thread, threads per row.
// 16-byte loads where the rows allow them, else pairs of 16-bit elements,
// else single ones; up to 32 elements a thread (their two sums of the
// backward pass take 64 registers), and never more than 512 threads a row.
struct Spread {
    int vec, cpt, lanes;
};

Spread spread_of(int esz, int64_t width, bool vec16, bool vec4)
{
    const int full = 16 / esz;
    Spread s;
    if (vec16) {
        s.vec = full;
        s.cpt = width <= 32 * full ? 1 : width <= 64 * full ? 2 : (esz == 2 || width <= 8192) ? 4 : 8;
    } else if (vec4 && esz == 2) {
        s.vec = 2;
        s.cpt = width <= 256 ? 4 : width <= 8192 ? 8 : 16;
    } else {
        s.vec = 1;
        s.cpt = width <= 128 ? 4 : width <= 8192 ? 16 : 32;
    }
    const int64_t per = static_cast<int64_t>(s.vec) * s.cpt;
    s.lanes = static_cast<int>(((width + per - 1) / per + 31) / 32 * 32);
    return s;
}

int64_t parts_of(int64_t rows_per_group, int64_t groups, bool warp, int lanes)
{
    const int64_t per_block = warp ? kRowsPerBlock : 1;
    const int64_t want = (rows_per_group + per_block - 1) / per_block;
    // Resident blocks: about 512 threads an SM (128 registers a thread).
    const int64_t per_sm = warp ? 2 : (lanes >= 512 ? 1 : 512 / lanes);
    int64_t cap = h3qk_internal_sm_count() * per_sm / groups;
    if (cap < 1) cap = 1;
    return want < cap ? want : cap;
}

// The spread a call could use at most parallel (for the size of the workspace,
// which is fixed before alignment is known).
int64_t max_parts(int64_t rows_per_group, int64_t groups)
{
    int64_t cap = h3qk_internal_sm_count() * static_cast<int64_t>(8) / groups;
    if (cap < 1) cap = 1;
    return rows_per_group < cap ? rows_per_group : cap;
}

template <typename T, int VEC, int CPT, bool WARP>
cudaError_t launch(bool backward, const LnArgs& a, int64_t groups, int lanes, cudaStream_t st)
{
    const int threads = WARP ? 32 * kRowsPerBlock : lanes;
    if (backward) {
        const dim3 grid(static_cast<unsigned>(a.parts), static_cast<unsigned>(groups));
        const size_t smem = WARP && a.partial ? static_cast<size_t>(kRowsPerBlock) * a.width * 4 : 0;
        layer_norm_backward_kernel<T, VEC, CPT, WARP><<<grid, threads, smem, st>>>(a);
    } else {
        const int64_t want = WARP ? (a.rows_per_group + kRowsPerBlock - 1) / kRowsPerBlock : a.rows_per_group;
        const int64_t cap = h3qk_internal_sm_count() * static_cast<int64_t>(2048 / threads);
        const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), static_cast<unsigned>(groups));
        layer_norm_kernel<T, VEC, CPT, WARP><<<grid, threads, 0, st>>>(a);
    }
    h3qk_internal_count_launch();
    return cudaGetLastError();
}

// Only the pairs that spread_of can choose are instantiated.
template <typename T, int FULL>
cudaError_t dispatch(bool back, const LnArgs& a, int64_t groups, const Spread& s, cudaStream_t st)
{
    const bool warp = s.lanes == 32;
    if (s.vec == FULL) {
        if (s.cpt == 1) return launch<T, FULL, 1, true>(back, a, groups, s.lanes, st);
        if (s.cpt == 2) return launch<T, FULL, 2, true>(back, a, groups, s.lanes, st);
        if constexpr (FULL == 4)
            if (s.cpt == 8) return launch<T, FULL, 8, false>(back, a, groups, s.lanes, st);
        if (warp) return launch<T, FULL, 4, true>(back, a, groups, s.lanes, st);
        return launch<T, FULL, 4, false>(back, a, groups, s.lanes, st);
    }
    if constexpr (FULL == 8) {
        if (s.vec == 2) {
            if (s.cpt == 4) return launch<T, 2, 4, true>(back, a, groups, s.lanes, st);
            if (s.cpt == 16) return launch<T, 2, 16, false>(back, a, groups, s.lanes, st);
            if (warp) return launch<T, 2, 8, true>(back, a, groups, s.lanes, st);
            return launch<T, 2, 8, false>(back, a, groups, s.lanes, st);
        }
    }
    if (s.cpt == 4) return launch<T, 1, 4, true>(back, a, groups, s.lanes, st);
    if (s.cpt == 32) return launch<T, 1, 32, false>(back, a, groups, s.lanes, st);
    if (warp) return launch<T, 1, 16, true>(back, a, groups, s.lanes, st);
    return launch<T, 1, 16, false>(back, a, groups, s.lanes, st);
}

cudaError_t dispatch_type(bool backward, int dtype, const LnArgs& a, int64_t groups, const Spread& s, cudaStream_t st)
{
    if (dtype == H3QK_FP16) return dispatch<F16, 8>(backward, a, groups, s, st);
    if (dtype == H3QK_BF16) return dispatch<BF16, 8>(backward, a, groups, s, st);
    return dispatch<F32, 4>(backward, a, groups, s, st);
}

// Checks common to both directions.
h3qk_status check_rows(int dtype, int64_t rows, int32_t width, int64_t groups, int64_t* stride)
{
    if (dtype != H3QK_FP16 && dtype != H3QK_BF16 && dtype != H3QK_FP32) return H3QK_ERR_INVALID_ARG;
    if (rows < 0 || width < 1 || width > kMaxWidth) return H3QK_ERR_INVALID_ARG;
    if (groups < 1 || groups > 65535 || rows % groups) return H3QK_ERR_INVALID_ARG;
    if (*stride == 0) *stride = width;
    if (*stride < width) return H3QK_ERR_INVALID_ARG;
    if (rows > 0 && *stride > (INT64_C(1) << 40) / rows) return H3QK_ERR_INVALID_ARG;
    return H3QK_OK;
}

bool multiple(const void* p, int64_t stride, int esz, int n)
{
    return aligned(p, n) && stride * esz % n == 0;
}

}  // namespace

extern "C" h3qk_status h3qk_layer_norm(const void* x, h3qk_dtype dtype, int64_t rows, int32_t width,
                                       int64_t row_stride, const float* weight, const float* bias, int64_t groups,
                                       float eps, void* out, float* stats, h3qk_stream_t stream)
{
    const h3qk_status s = check_rows(dtype, rows, width, groups, &row_stride);
    if (s != H3QK_OK) return s;
    if (!(eps >= 0.0f) || eps > 3.0e38f) return H3QK_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !out || !stats)) return H3QK_ERR_INVALID_ARG;
    const int esz = dtype == H3QK_FP32 ? 4 : 2;
    if (!aligned(x, esz) || !aligned(out, esz) || !aligned(stats, 8) || !aligned(weight, 4) || !aligned(bias, 4))
        return H3QK_ERR_MISALIGNED;
    const Range ins[3] = {range_of(x, rows > 0 ? ((rows - 1) * row_stride + width) * esz : 0),
                          range_of(weight, weight ? groups * width * 4 : 0),
                          range_of(bias, bias ? groups * width * 4 : 0)};
    const Range outs[2] = {range_of(out, rows * width * esz), range_of(stats, rows * 8)};
    if (overlap(outs[0], outs[1])) return H3QK_ERR_ALIAS;
    for (const Range& o : outs)
        for (const Range& i : ins)
            if (overlap(o, i)) return H3QK_ERR_ALIAS;
    if (rows == 0) return H3QK_OK;
    LnArgs a = {};
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.stats = stats;
    a.out = out;
    a.rows_per_group = rows / groups;
    a.x_stride = row_stride;
    a.out_stride = width;
    a.width = width;
    a.eps = eps;
    a.inv_width = 1.0f / static_cast<float>(width);
    const bool v16 = multiple(x, row_stride, esz, 16) && multiple(out, width, esz, 16) && aligned(weight, 16) && aligned(bias, 16);
    const bool v4 = multiple(x, row_stride, esz, 4) && multiple(out, width, esz, 4) && width % 2 == 0;
    return status_of(dispatch_type(false, dtype, a, groups, spread_of(esz, width, v16, v4),
                                   reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" size_t h3qk_layer_norm_backward_workspace_bytes(int64_t rows, int32_t width, int64_t groups)
{
    if (rows < 0 || width < 1 || width > kMaxWidth || groups < 1 || groups > 65535 || rows % groups) return 0;
    return static_cast<size_t>(groups * max_parts(rows / groups, groups)) * 2 * width * 4;
}

extern "C" h3qk_status h3qk_layer_norm_backward(const void* grad_out, int64_t grad_stride, const void* x,
                                                h3qk_dtype dtype, int64_t rows, int32_t width, int64_t row_stride,
                                                const float* weight, int64_t groups, const float* stats,
                                                void* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                                                size_t workspace_bytes, h3qk_stream_t stream)
{
    h3qk_status s = check_rows(dtype, rows, width, groups, &row_stride);
    if (s == H3QK_OK) s = check_rows(dtype, rows, width, groups, &grad_stride);
    if (s != H3QK_OK) return s;
    if (rows > 0 && (!grad_out || !x || !stats || !grad_x)) return H3QK_ERR_INVALID_ARG;
    const bool sums = grad_weight || grad_bias;
    const size_t need = sums ? h3qk_layer_norm_backward_workspace_bytes(rows, width, groups) : 0;
    if (need && (!workspace || workspace_bytes < need)) return H3QK_ERR_INVALID_ARG;
    const int esz = dtype == H3QK_FP32 ? 4 : 2;
    if (!aligned(x, esz) || !aligned(grad_out, esz) || !aligned(grad_x, esz) || !aligned(stats, 8) ||
        !aligned(weight, 4) || !aligned(grad_weight, 4) || !aligned(grad_bias, 4) || (need && !aligned(workspace, 16)))
        return H3QK_ERR_MISALIGNED;
    const int64_t wbytes = groups * width * 4;
    const Range ins[4] = {range_of(x, rows > 0 ? ((rows - 1) * row_stride + width) * esz : 0),
                          range_of(grad_out, rows > 0 ? ((rows - 1) * grad_stride + width) * esz : 0),
                          range_of(weight, weight ? wbytes : 0), range_of(stats, rows * 8)};
    const Range outs[4] = {range_of(grad_x, rows * width * esz), range_of(grad_weight, grad_weight ? wbytes : 0),
                           range_of(grad_bias, grad_bias ? wbytes : 0), range_of(workspace, need)};
    for (int i = 0; i < 4; ++i) {
        for (int k = i + 1; k < 4; ++k)
            if (overlap(outs[i], outs[k])) return H3QK_ERR_ALIAS;
        for (const Range& in : ins)
            if (overlap(outs[i], in)) return H3QK_ERR_ALIAS;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LnArgs a = {};
    a.x = x;
    a.dy = grad_out;
    a.weight = weight;
    a.stats = const_cast<float*>(stats);
    a.out = grad_x;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    a.rows_per_group = rows / groups;
    a.x_stride = row_stride;
    a.dy_stride = grad_stride;
    a.out_stride = width;
    a.width = width;
    a.inv_width = 1.0f / static_cast<float>(width);
    if (rows > 0) {
        const bool v16 = multiple(x, row_stride, esz, 16) && multiple(grad_out, grad_stride, esz, 16) &&
                         multiple(grad_x, width, esz, 16) && aligned(weight, 16);
        const bool v4 = multiple(x, row_stride, esz, 4) && multiple(grad_out, grad_stride, esz, 4) &&
                        multiple(grad_x, width, esz, 4) && width % 2 == 0;
        const Spread sp = spread_of(esz, width, v16, v4);
        const int64_t most = max_parts(a.rows_per_group, groups);
        const int64_t parts = parts_of(a.rows_per_group, groups, sp.lanes == 32, sp.lanes);
        a.parts = static_cast<int32_t>(parts < most ? parts : most);
        const cudaError_t e = dispatch_type(true, dtype, a, groups, sp, st);
        if (e != cudaSuccess) return h3qk_internal_fail_cuda(e);
    }
    if (!sums) return H3QK_OK;
    const dim3 grid((width + kSumCols - 1) / kSumCols, static_cast<unsigned>(groups), 2);
    return status_of(launch_chained(sum_parts_kernel, grid, dim3(kSumCols, kSumLanes), 0, st,
                                    static_cast<const float*>(workspace), grad_weight, grad_bias,
                                    static_cast<int>(rows > 0 ? a.parts : 0), static_cast<int>(width)));
}
