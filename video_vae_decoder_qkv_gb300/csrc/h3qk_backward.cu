// The gradient of the fused QK preparation: from the gradients of Q, K and V
// (head-major or token-major) to the gradient of the packed projection rows
// and of the two norm weights.  Per head row, with R the rotation and
// xh = x inv, inv = (sum x^2 / D + eps)^-1/2 (the forward's 16-bit rounding
// points count as the identity):
//   dn = R^T dy (the rotation by minus the angle),  dw = sum dn xh,
//   g = dn w,  dx = inv (g - xh mean(g xh));   V: dx = dy.
//
// Bound by HBM: 16 bytes of x, dy and dx per 8 channels of Q and K, 32 per 8
// of V, and about 120 instructions a warp for 32 such chunks, a third of the
// memory time: 32,640 rows of 40 heads of 128 in bf16 take 0.43 ms, 6.2 TB/s.
// (Each head's loads are issued one head ahead; without that 0.51 ms.)  The
// layout is the forward's: a lane owns 8 channels, the
// lanes of a head row are a power of two, a warp holds 32 / lanes consecutive
// token rows of one head.  sum x^2 and sum g x do not depend on one another,
// so one pass of shuffles carries both.  The angles' cosines and sines are
// found once per token row and reused for the heads of the item.  The weight
// gradients stay in each lane's registers over all its rows; blocks write
// partial sums and a chained kernel adds them in a fixed order.
#include "h3qk_kernels.cuh"
#include "h3qk_ops.cuh"

namespace {

using namespace h3qk_ops;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

constexpr int kWarps = 8;

struct GradArgs {
    h3qk::Params p;           // the forward's description of the rows
    const uint16_t* grad[3];  // gradients of Q, K, V
    uint16_t* dx;             // [tokens, 3 H D]
    float* partial;           // [blocks][2][D]
    int64_t groups;           // groups of 32 / LPR token rows
    int32_t slices, slice_heads;
};

__device__ __forceinline__ uint4 load_stream(const uint16_t* p)
{
    return __ldcs(reinterpret_cast<const uint4*>(p));
}

template <bool BF16>
__device__ __forceinline__ void widen8(float (&o)[8], const uint4& v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = h3qk::widen2<BF16>(w[i]);
        o[2 * i] = f.x;
        o[2 * i + 1] = f.y;
    }
}

template <bool BF16, int LPR>
__global__ void __launch_bounds__(32 * kWarps, 2) prepare_backward_kernel(const __grid_constant__ GradArgs a)
{
    __shared__ float merge[kWarps][2][8][32];
    allow_dependents();
    const h3qk::Params& p = a.p;
    constexpr int TPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = lane % LPR, sub = lane / LPR;
    const bool in = c < p.chunks;
    const int D = p.head_dim;
    const float inv_d = 1.0f / static_cast<float>(D);
    float w[2][8], dw[2][8];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[t][i] = in ? __ldg((t ? p.wk : p.wq) + 8 * c + i) : 0.0f;
            dw[t][i] = 0.0f;
        }
    const int64_t items = a.groups * a.slices;
    const int64_t HD = static_cast<int64_t>(p.heads) * D;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kWarps + warp; it < items;
         it += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t group = it / a.slices;
        const int h0 = static_cast<int>(it - group * a.slices) * a.slice_heads;
        const int h1 = min(h0 + a.slice_heads, p.heads);
        const int64_t r = group * TPW + sub;
        const bool row = in && r < p.rows;
        const int64_t b = r / p.seq, s = r - b * p.seq;
        int64_t valid = p.valid_len;
        if (p.valid_lens && row) valid = min(max(static_cast<int64_t>(__ldg(p.valid_lens + b)), int64_t{0}), p.seq);
        const bool live = row && s < valid;
        uint16_t* out = a.dx + r * 3 * HD + 8 * c;
        float cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cs[i] = 1.0f;
            sn[i] = 0.0f;
            const int pair = 4 * c + i;
            if (live && 2 * pair < p.rotary_dim) {
                const float pos = static_cast<float>(__ldg(p.pos + r * p.n_axes + p.axis[pair]));
                h3qk::sincos_h3(__fmul_rn(pos, p.inv_freq[pair]), sn[i], cs[i]);
            }
        }
        const uint16_t* x = p.qkv + r * p.row_stride + 8 * c;
        const int64_t gbase = b * p.out_bstride + s * p.out_sstride + 8 * c;
        // The next head's five loads are on their way while this one is computed.
        uint4 nx[2] = {}, ng[3] = {};
        auto fetch = [&](int h) {
            if (live && h < h1) {
                const int64_t go = gbase + h * p.out_hstride;
                nx[0] = load_stream(x + h * D);
                nx[1] = load_stream(x + HD + h * D);
#pragma unroll
                for (int t = 0; t < 3; ++t) ng[t] = load_stream(a.grad[t] + go);
            }
        };
        fetch(h0);
        for (int h = h0; h < h1; ++h) {
            const uint4 xv[2] = {nx[0], nx[1]}, gv[3] = {ng[0], ng[1], ng[2]};
            fetch(h + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float xf[8], dn[8];
                widen8<BF16>(xf, xv[t]);
                widen8<BF16>(dn, gv[t]);
                float ss = 0.0f, gx = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = dn[2 * i], v = dn[2 * i + 1];
                    dn[2 * i] = fmaf(v, sn[i], u * cs[i]);
                    dn[2 * i + 1] = fmaf(-u, sn[i], v * cs[i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(xf[i], xf[i], ss);
                    gx = fmaf(dn[i] * w[t][i], xf[i], gx);
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) {
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    gx += __shfl_xor_sync(0xffffffffu, gx, o);
                }
                const float inv = 1.0f / sqrtf(ss * inv_d + p.eps);
                // xh and this mean stay near 1 for rows of any size; inv^3 would not.
                const float mean = inv * gx * inv_d;
                uint32_t ow[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float o[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int e = 2 * i + j;
                        const float xh = xf[e] * inv;
                        if (live) dw[t][e] = fmaf(dn[e], xh, dw[t][e]);
                        o[j] = inv * fmaf(-mean, xh, dn[e] * w[t][e]);
                    }
                    ow[i] = live ? h3qk::round2<BF16>(o[0], o[1]) : 0u;
                }
                if (row) __stcs(reinterpret_cast<uint4*>(out + t * HD + h * D), make_uint4(ow[0], ow[1], ow[2], ow[3]));
            }
            if (row) __stcs(reinterpret_cast<uint4*>(out + 2 * HD + h * D), gv[2]);
        }
    }
    // Lanes with the same channels: the warp's token rows, then the block's warps.
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = dw[t][i];
#pragma unroll
            for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            merge[warp][t][i][lane] = v;
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += blockDim.x) {
        const int t = e / D, d = e - t * D;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) v += merge[q][t][d % 8][d / 8];
        a.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + e] = v;
    }
}

// grad_w[t][d] = the sum of the blocks' partial rows: one block per 32
// channels, 32 lanes of blocks, each adding its share in order.
__global__ void sum_weight_grads_kernel(const float* partial, float* grad_wq, float* grad_wk, int blocks, int D)
{
    __shared__ float s[32][33];
    wait_for_previous();
    const int e = blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (e < 2 * D)
        for (int b = threadIdx.y; b < blocks; b += 32) v += partial[static_cast<int64_t>(b) * 2 * D + e];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    v = warp_sum(s[threadIdx.x][threadIdx.y]);
    const int o = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && o < 2 * D) {
        float* dst = o < D ? grad_wq : grad_wk;
        if (dst) dst[o < D ? o : o - D] = v;
    }
}

template <bool BF16>
cudaError_t launch_backward(int P, const GradArgs& a, int blocks, cudaStream_t st)
{
    switch (P) {
    case 1: prepare_backward_kernel<BF16, 1><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    case 2: prepare_backward_kernel<BF16, 2><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    case 4: prepare_backward_kernel<BF16, 4><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    case 8: prepare_backward_kernel<BF16, 8><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    case 16: prepare_backward_kernel<BF16, 16><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    default: prepare_backward_kernel<BF16, 32><<<blocks, 32 * kWarps, 0, st>>>(a); break;
    }
    h3qk_internal_count_launch();
    return cudaGetLastError();
}

// Blocks of a call: two resident per SM (the register bound above).
int block_cap() { return 2 * h3qk_internal_sm_count(); }

}  // namespace

extern "C" size_t h3qk_prepare_backward_workspace_bytes(int32_t head_dim)
{
    if (head_dim < 8 || head_dim > 256 || head_dim % 8) return 0;
    return static_cast<size_t>(block_cap()) * 2 * head_dim * 4;
}

extern "C" h3qk_status h3qk_prepare_backward(const void* grad_q, const void* grad_k, const void* grad_v,
                                             const void* qkv, const float* norm_wq, const float* norm_wk,
                                             const int32_t* positions, int64_t tokens, int32_t heads,
                                             int32_t head_dim, int32_t rotary_dim, int64_t valid_len,
                                             void* grad_qkv, float* grad_wq, float* grad_wk, void* workspace,
                                             size_t workspace_bytes, const h3qk_opts* opts, h3qk_stream_t stream)
{
    h3qk_opts o;
    h3qk_opts_init(&o);
    if (opts) o = *opts;
    h3qk_detail::Plan pl;
    const h3qk_status s = h3qk_detail::plan_inputs(qkv, norm_wq, norm_wk, positions, tokens, heads, head_dim,
                                                   rotary_dim, valid_len, H3QK_BF16, o, stream, &pl);
    if (s != H3QK_OK) return s;
    if (tokens > 0 && (!grad_q || !grad_k || !grad_v || !grad_qkv)) return H3QK_ERR_INVALID_ARG;
    const size_t need = h3qk_prepare_backward_workspace_bytes(head_dim);
    if (!workspace || workspace_bytes < need) return H3QK_ERR_INVALID_ARG;
    if (!aligned(grad_q, 16) || !aligned(grad_k, 16) || !aligned(grad_v, 16) || !aligned(grad_qkv, 16) ||
        !aligned(workspace, 16) || !aligned(grad_wq, 4) || !aligned(grad_wk, 4))
        return H3QK_ERR_MISALIGNED;
    const int64_t n = tokens * pl.HD * 2;
    const Range grads[3] = {range_of(grad_q, n), range_of(grad_k, n), range_of(grad_v, n)};
    const Range outs[4] = {range_of(grad_qkv, 3 * n), range_of(grad_wq, grad_wq ? head_dim * 4 : 0),
                           range_of(grad_wk, grad_wk ? head_dim * 4 : 0), range_of(workspace, need)};
    for (int i = 0; i < 4; ++i) {
        for (int k = i + 1; k < 4; ++k)
            if (overlap(outs[i], outs[k])) return H3QK_ERR_ALIAS;
        for (const Range& g : grads)
            if (overlap(outs[i], g)) return H3QK_ERR_ALIAS;
        if (h3qk_detail::overlaps_inputs(pl, outs[i])) return H3QK_ERR_ALIAS;
    }
    int blocks = 0;
    if (tokens > 0) {
        GradArgs a;
        a.p = pl.p;
        a.grad[0] = static_cast<const uint16_t*>(grad_q);
        a.grad[1] = static_cast<const uint16_t*>(grad_k);
        a.grad[2] = static_cast<const uint16_t*>(grad_v);
        a.dx = static_cast<uint16_t*>(grad_qkv);
        a.partial = static_cast<float*>(workspace);
        const int tpw = 32 / pl.P;
        a.groups = (tokens + tpw - 1) / tpw;
        // Heads are cut into slices of h: a warp's turns times a slice's cost,
        // h heads and the rows' angles (about two thirds of a head's work), is
        // least.  It keeps the last turn full: 8 x 4896 rows of 16 heads of 64
        // in two slices are 8.05 turns.
        const int64_t warps = static_cast<int64_t>(block_cap()) * kWarps;
        int64_t least = INT64_MAX;
        for (int32_t h = heads; h >= 1; --h) {
            const int64_t slices = (heads + h - 1) / h;
            if (slices > 64) break;
            const int64_t cost = (a.groups * slices + warps - 1) / warps * (3 * static_cast<int64_t>(h) + 2);
            if (cost < least) {
                least = cost;
                a.slice_heads = h;
                a.slices = static_cast<int32_t>(slices);
            }
        }
        const int64_t want = (a.groups * a.slices + kWarps - 1) / kWarps;
        blocks = static_cast<int>(want < block_cap() ? want : block_cap());
        const cudaError_t e = pl.bf16 ? launch_backward<true>(pl.P, a, blocks, pl.st)
                                      : launch_backward<false>(pl.P, a, blocks, pl.st);
        if (e != cudaSuccess) return h3qk_internal_fail_cuda(e);
    }
    if (!grad_wq && !grad_wk) return H3QK_OK;
    return status_of(launch_chained(sum_weight_grads_kernel, dim3((2 * head_dim + 31) / 32), dim3(32, 32), 0, pl.st,
                                    static_cast<const float*>(workspace), grad_wq, grad_wk, blocks,
                                    static_cast<int>(head_dim)));
}
