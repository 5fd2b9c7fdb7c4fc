// Attention forward, few rows (a token or a few per request over a cache).
//
// Bound by reading the cache once.  All query rows that share a K/V head
// (`group` heads x q_rows) form one tile of 16, so K and V are read once for
// the group.  The keys are cut into chunks, a block of four warps each; each
// warp takes 16 keys at a time, keeps its own running maximum, sum and O, and
// the warps meet in shared memory once at the end.  A second, chained kernel
// joins the chunks.
//
// K and V go from global memory into the fragments of the 16 x 8 x 16
// product, 16 bytes a load: the contraction over
// channels may be taken in any order, so a lane's 8 neighbouring channels of
// a key serve two steps if Q is held in the same order; and the columns of O
// may come in any order, so a lane's 8 neighbouring channels of two keys
// become (key, key + 1) pairs with one byte permute each.  The loads run ahead
// as asynchronous copies; each lane copies just the 16-byte pieces it will use
// itself, into slots of its own, so there is nothing to synchronise and no
// bank conflict.  The tensor work is
// a few percent of the load time, so the older warp-wide product does here;
// tcgen05's 128 rows would be nearly empty.
// 32 caches of 32,768 keys, 8 K/V heads of 128, bf16: 0.74 ms, 5.8 TB/s; with
// the loads straight into registers and not ahead it was 0.84.
#include "h3qk_attn.cuh"

namespace {

using namespace h3qk_tc;
using h3qk_core::Bend;
using h3qk_core::Params;
using h3qk_core::Stretch;

constexpr int kWarps = 4;
constexpr int kRows = 16;

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kAhead = 3;  // turns of 16 keys a warp has in flight or in use

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint4* dst, const uint16_t* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The floats one block leaves for the join: per row O[dim], m, sum.
__host__ __device__ inline int64_t part_floats(int dim) { return static_cast<int64_t>(kRows) * (dim + 2); }

// Writes one joined row.
template <bool BF16>
__device__ __forceinline__ void finish_lse(const Params& p, int item, int head, int row, float m, float sum, float shift)
{
    p.lse[(static_cast<int64_t>(item) * p.heads + head) * p.q_rows + row] =
        sum == 0.0f ? -INFINITY : (m - shift + log2f(sum)) * h3qk_core::kLn2;
}

// DH: blocks of 64 channels.
template <bool BF16, int DH>
__global__ void __launch_bounds__(32 * kWarps) attention_split_kernel(const __grid_constant__ Params p)
{
    constexpr int NB = 2 * DH;
    constexpr float kShift = BF16 ? 0.0f : 7.0f;
    // [warp][turn][piece][lane]: K 2 x NB pieces, V 4 x DH; at the end the warps' O
    constexpr int kPieces = 2 * NB + 4 * DH;
    extern __shared__ __align__(16) uint8_t dynamic[];
    auto& slots = *reinterpret_cast<uint4(*)[kWarps][kAhead][kPieces][32]>(dynamic);
    float(*sh_o)[kRows][64 * DH + 4] = reinterpret_cast<float(*)[kRows][64 * DH + 4]>(slots);
    static_assert(sizeof(slots) >= kWarps * kRows * (64 * DH + 4) * 4, "the warps' O fits the slots");
    __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows];
    h3qk_ops::allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & 3, g = lane >> 2;
    const int kv = blockIdx.y % p.kv_heads, rt = blockIdx.y / p.kv_heads;
    const int tiles = gridDim.y / p.kv_heads;
    Stretch s;
    h3qk_core::find_stretch(s, p, 0, blockIdx.z, 1, false);
    const int all = p.group * p.q_rows;

    const bool capped = p.cap > 0.0f;

    // The two rows of this lane.
    int lim[2], head[2], row[2];
    bool has[2];
    int at[2];  // positions among the keys
    Bend bend[2];
    int most = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = rt * kRows + g + 8 * h;
        has[h] = t < all;
        head[h] = kv * p.group + (has[h] ? t / p.q_rows : 0);
        row[h] = has[h] ? t % p.q_rows : 0;
        lim[h] = has[h] && row[h] < s.rows ? max(h3qk_core::limit_of(s, p.causal, row[h]), 0) : 0;
        most = max(most, lim[h]);
        at[h] = s.start + row[h];
        bend[h] = h3qk_core::bend_of(p, head[h]);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    const int k_first = blockIdx.x * p.chunk;
    const int k_end = min(k_first + p.chunk, most);

    float o[8 * DH][4];
#pragma unroll
    for (int t = 0; t < 8 * DH; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    if (k_first + 16 * warp < k_end) {
        uint4 q[2][NB];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const int d = 32 * b + 8 * c;
                q[h][b] = make_uint4(0, 0, 0, 0);
                if (has[h] && d < p.dim)
                    q[h][b] = __ldg(reinterpret_cast<const uint4*>(p.q + s.item * p.qs.item + head[h] * p.qs.head +
                                                                   row[h] * p.qs.row + d));
            }
        const uint16_t* kp = p.k + s.item * p.ks.item + kv * p.ks.head + 8 * c;
        const uint16_t* vp = p.v + s.item * p.vs.item + kv * p.vs.head + 8 * g;
        auto fetch = [&](int j, int turn) {
            uint4(*to)[32] = slots[warp][turn];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int key = j + 8 * t + g;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const bool there = key < k_end && 32 * b + 8 * c < p.dim;
                    copy16(&to[t * NB + b][lane], there ? kp + key * p.ks.row + 32 * b : kp, there);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int key = j + 2 * c + (t & 1) + 8 * (t >> 1);
#pragma unroll
                for (int b = 0; b < DH; ++b) {
                    const bool there = key < k_end && 64 * b + 8 * g < p.dim;
                    copy16(&to[2 * NB + t * DH + b][lane], there ? vp + key * p.vs.row + 64 * b : vp, there);
                }
            }
        };
        int j = k_first + 16 * warp;
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) {
            if (j + i * 16 * kWarps < k_end) fetch(j + i * 16 * kWarps, i);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int turn = 0;
        for (; j < k_end; j += 16 * kWarps) {
            const int next = j + (kAhead - 1) * 16 * kWarps;
            if (next < k_end) fetch(next, turn == 0 ? kAhead - 1 : turn - 1);
            asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
            uint4 kr[2][NB], vr[4][DH];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b) kr[t][b] = slots[warp][turn][t * NB + b][lane];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int b = 0; b < DH; ++b) vr[t][b] = slots[warp][turn][2 * NB + t * DH + b][lane];
            turn = turn + 1 == kAhead ? 0 : turn + 1;
            float sc[2][4] = {};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    mma16<BF16>(sc[t], q[0][b].x, q[1][b].x, q[0][b].y, q[1][b].y, kr[t][b].x, kr[t][b].y);
                    mma16<BF16>(sc[t], q[0][b].z, q[1][b].z, q[0][b].w, q[1][b].w, kr[t][b].z, kr[t][b].w);
                }
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = m[h];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float small[2];
                    if (capped) {
                        const uint64_t raw = pair(sc[t][2 * h], sc[t][2 * h + 1]), z = mul_pair(raw, pair(bend[h].in, bend[h].in));
                        const uint64_t flat = mul_pair(raw, pair(bend[h].plain, bend[h].plain));
                        unpair(small[0], small[1], mul_pair(flat, h3qk_core::tanh_series(mul_pair(z, z))));
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int key = j + 8 * t + 2 * c + e;
                        float v = sc[t][2 * h + e] * bend[h].in;
                        if (capped) {
                            const float bent = fmaf(-2.0f * bend[h].cap, rcp_fast(exp2_fast(v) + 1.0f), bend[h].cap);
                            v = fabsf(v) < h3qk_core::kSmall ? small[e] : bent;
                        }
                        v = fmaf(-bend[h].slope, fabsf(static_cast<float>(at[h] - key)), v);
                        v = key < lim[h] ? v : -INFINITY;
                        sc[t][2 * h + e] = v;
                        top = fmaxf(top, v);
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                f[h] = top == -INFINITY ? 1.0f : exp2_fast(m[h] - top);
                m[h] = top;
                const float off = (top == -INFINITY ? 0.0f : top) - kShift;
                float add = 0.0f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float pv = exp2_fast(sc[t][2 * h + e] - off);
                        sc[t][2 * h + e] = pv;
                        add += pv;
                    }
                l[h] = fmaf(l[h], f[h], add);
            }
            if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                for (int t = 0; t < 8 * DH; ++t) {
                    o[t][0] *= f[0];
                    o[t][1] *= f[0];
                    o[t][2] *= f[1];
                    o[t][3] *= f[1];
                }
            }
            const uint32_t a0 = round_pair<BF16>(sc[0][0], sc[0][1]), a1 = round_pair<BF16>(sc[0][2], sc[0][3]);
            const uint32_t a2 = round_pair<BF16>(sc[1][0], sc[1][1]), a3 = round_pair<BF16>(sc[1][2], sc[1][3]);
#pragma unroll
            for (int b = 0; b < DH; ++b)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const uint32_t sel = (t & 1) ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(word(vr[0][b], t / 2), word(vr[1][b], t / 2), sel);
                    const uint32_t b1 = __byte_perm(word(vr[2][b], t / 2), word(vr[3][b], t / 2), sel);
                    mma16<BF16>(o[8 * b + t], a0, a1, a2, a3, b0, b1);
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
    }

    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    // Join the block's warps.  Column n = 2c + e of product t of block b is
    // channel 64 b + 8 n + t.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int b = 0; b < DH; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < 8; t += 4)
                    *reinterpret_cast<float4*>(&sh_o[warp][g + 8 * h][64 * b + 8 * (2 * c + e) + t]) =
                        make_float4(o[8 * b + t][2 * h + e], o[8 * b + t + 1][2 * h + e], o[8 * b + t + 2][2 * h + e],
                                    o[8 * b + t + 3][2 * h + e]);
        if (c == 0) {
            sh_m[warp][g + 8 * h] = m[h];
            sh_l[warp][g + 8 * h] = l[h];
        }
    }
    __syncthreads();
    const int per = p.dim / 4;
    float* part = p.part + ((static_cast<int64_t>(blockIdx.z) * p.kv_heads + kv) * tiles + rt) * p.splits * part_floats(p.dim) +
                  blockIdx.x * part_floats(p.dim);
    for (int i = threadIdx.x; i < kRows * per; i += 32 * kWarps) {
        const int r = i / per, d = 4 * (i - r * per);
        const int t = rt * kRows + r;
        if (t >= all) break;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][r]);
        float sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sh_m[w][r] == -INFINITY && !(sh_l[w][r] != sh_l[w][r]) ? 0.0f : exp2_fast(sh_m[w][r] - top);
            const float4 x = *reinterpret_cast<const float4*>(&sh_o[w][r][d]);
            sum = fmaf(sh_l[w][r], f, sum);
            v.x = fmaf(x.x, f, v.x);
            v.y = fmaf(x.y, f, v.y);
            v.z = fmaf(x.z, f, v.z);
            v.w = fmaf(x.w, f, v.w);
        }
        if (p.splits == 1) {
            const int hd = kv * p.group + t / p.q_rows, rw = t % p.q_rows;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            uint2 w;
            w.x = round_pair<BF16>(v.x * inv, v.y * inv);
            w.y = round_pair<BF16>(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2*>(p.out + s.item * p.os.item + hd * p.os.head + rw * p.os.row + d) = w;
            if (d == 0) finish_lse<BF16>(p, s.item, hd, rw, top, sum, kShift);
        } else {
            if (k_first < k_end) *reinterpret_cast<float4*>(part + r * p.dim + d) = v;
            if (d == 0) *reinterpret_cast<float2*>(part + kRows * p.dim + 2 * r) = make_float2(top, sum);
        }
    }
}

// One block a row: each warp joins every fourth chunk, in order, then the
// block joins its warps.
template <bool BF16>
__global__ void __launch_bounds__(32 * kWarps) join_split_kernel(const __grid_constant__ Params p)
{
    constexpr float kShift = BF16 ? 0.0f : 7.0f;
    __shared__ float4 sh_v[kWarps][32];
    __shared__ float sh_sum[kWarps], sh_top[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int all = p.group * p.q_rows;
    const int tiles = (all + kRows - 1) / kRows;
    const int t = static_cast<int>(blockIdx.x % all);
    const int kv = static_cast<int>(blockIdx.x / all % p.kv_heads);
    const int item = static_cast<int>(blockIdx.x / all / p.kv_heads);
    const int64_t size = part_floats(p.dim);
    const float* part = p.part + ((static_cast<int64_t>(item) * p.kv_heads + kv) * tiles + t / kRows) * p.splits * size;
    const int in = t % kRows, d = 4 * lane;
    h3qk_ops::wait_for_previous();
    auto stat = [&](int sp) { return __ldcg(reinterpret_cast<const float2*>(part + sp * size + kRows * p.dim + 2 * in)); };
    float top = -INFINITY;
    for (int sp = threadIdx.x; sp < p.splits; sp += 32 * kWarps) top = fmaxf(top, stat(sp).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) sh_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWarps; ++q) top = fmaxf(top, sh_top[q]);
    float sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < p.splits; s0 += 32 * kWarps) {
        const int mine_at = s0 + lane * kWarps + warp;
        float2 mine = make_float2(-INFINITY, 0.0f);
        if (mine_at < p.splits) mine = stat(mine_at);
        // a chunk without visible keys left no O; a NaN sum is passed on
        const float f = mine.y == 0.0f ? 0.0f : exp2_fast(mine.x - top);
        const int n = min(32, (p.splits - s0 - warp + kWarps - 1) / kWarps);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float fi = __shfl_sync(0xffffffffu, f, i);
            const float li = __shfl_sync(0xffffffffu, mine.y, i);
            sum = fmaf(li, fi, sum);
            if (d < p.dim && li != 0.0f) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(part + (s0 + i * kWarps + warp) * size + in * p.dim + d));
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
    for (int q = 1; q < kWarps; ++q) {
        const float4 x = sh_v[q][lane];
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
        sum += sh_sum[q];
    }
    const int head = kv * p.group + t / p.q_rows, row = t % p.q_rows;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (d < p.dim) {
        uint2 w;
        w.x = round_pair<BF16>(v.x * inv, v.y * inv);
        w.y = round_pair<BF16>(v.z * inv, v.w * inv);
        *reinterpret_cast<uint2*>(p.out + item * p.os.item + head * p.os.head + row * p.os.row + d) = w;
    }
    if (lane == 0) finish_lse<BF16>(p, item, head, row, top, sum, kShift);
}

template <bool BF16, int DH>
cudaError_t launch_split(const Params& p, dim3 grid, cudaStream_t st)
{
    constexpr int smem = kWarps * kAhead * 8 * DH * 512;
    auto* kernel = attention_split_kernel<BF16, DH>;
    static bool raised[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!raised[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        raised[dev] = true;
    }
    kernel<<<grid, 32 * kWarps, smem, st>>>(p);
    h3qk_internal_count_launch();
    return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch(const Params& p, cudaStream_t st)
{
    const int all = p.group * p.q_rows;
    const dim3 grid(p.splits, p.kv_heads * ((all + kRows - 1) / kRows), p.batch);
    const cudaError_t e = p.dim <= 64 ? launch_split<BF16, 1>(p, grid, st) : launch_split<BF16, 2>(p, grid, st);
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(p.batch) * p.kv_heads * all;
    return h3qk_ops::launch_chained(join_split_kernel<BF16>, dim3(static_cast<unsigned>(rows)), dim3(32 * kWarps), 0, st, p);
}

}  // namespace

cudaError_t h3qk_core::forward_split(bool bf16, const Params& p, cudaStream_t st)
{
    return bf16 ? launch<true>(p, st) : launch<false>(p, st);
}
