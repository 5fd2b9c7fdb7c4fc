// Layer norm and its gradient.
//   mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
//   xh = (x - mean) rstd,  y = xh w + b
//   g = dy w,  dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both directions are bound by HBM: each element crosses it once each way.
// Rows come in asynchronously a few ahead of their use, since a row's two
// reductions leave the memory idle otherwise.  A row of up to 512 columns
// belongs to one warp (eight rows a block, shuffles only); a longer one to a
// block of its own.  Blocks walk many rows with every thread on fixed
// columns, so weights are read once and stay in registers.  65,280 rows of
// 5,120 in bf16: forward 0.25 ms (5.4 TB/s), backward 0.35 ms (5.8 TB/s);
// loading each row when its turn came, they took 0.36 and 0.53.  Rows off
// 16-byte boundaries cost more instructions than bytes: 2 to 4 TB/s in pairs,
// 1.5 to 3 in single 16-bit elements.
// The variance is the sum of squared deviations from the mean just found,
// not E[x^2] - mean^2, which loses all digits where |mean| >> deviation.
//
// The weight gradient is a sum over all rows.  A block walks its rows with
// every thread on fixed columns, so dw and db grow in registers; each block
// then writes one partial row and a second, chained kernel adds the partial
// rows in a fixed order: no atomics, the same bits on every run.
#include "h3qk_ops.cuh"
#include "h3qk_tc.cuh"

#include <type_traits>

namespace {

using namespace h3qk_ops;
using h3qk_detail::aligned;
using h3qk_detail::overlap;
using h3qk_detail::Range;
using h3qk_detail::range_of;

constexpr int kMaxWidth = 16384;  // 512 threads of 32 elements
constexpr int kRowsPerBlock = 8;  // warp-per-row blocks

using h3qk_tc::add_pair;
using h3qk_tc::fma_pair;
using h3qk_tc::mul_pair;
using h3qk_tc::pair;
using h3qk_tc::unpair;

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

// Two elements as stored.
template <typename T>
using Word = std::conditional_t<sizeof(typename T::raw) == 2, uint32_t, uint64_t>;

// Two elements in binary32 (arithmetic is on such pairs: the packed
// instructions round each half on its own).
template <typename T>
__device__ __forceinline__ uint64_t widen(Word<T> v)
{
    if constexpr (sizeof(v) == 8) {
        return v;
    } else {
        const float2 f = h3qk_tc::widen_pair<T::kBf16>(v);
        return pair(f.x, f.y);
    }
}

template <typename T>
__device__ __forceinline__ Word<T> narrow(uint64_t v)
{
    if constexpr (sizeof(Word<T>) == 8) {
        return v;
    } else {
        float lo, hi;
        unpair(lo, hi, v);
        return h3qk_tc::round_pair<T::kBf16>(lo, hi);
    }
}

// What one thread holds of a row: CPT chunks of VEC neighbouring elements,
// lanes * VEC columns apart, as pairs.  With single elements a pair is two chunks.
template <typename T, int VEC, int CPT>
struct Slice {
    static constexpr int kElems = VEC * CPT, kPairs = kElems / 2;
    static constexpr int kChunkBytes = VEC * static_cast<int>(sizeof(typename T::raw));
    static_assert(kElems % 2 == 0, "elements go in pairs");
    using Raw = typename T::raw;
    int lanes, lane, width;

    __device__ __forceinline__ int column(int e) const { return (e / VEC * lanes + lane) * VEC + e % VEC; }
    __device__ __forceinline__ bool has(int k) const { return (k * lanes + lane) * VEC < width; }

    static __device__ __forceinline__ void put(Word<T> (&w)[kPairs], int k, const uint4& v)
    {
        if constexpr (sizeof(Word<T>) == 4) {
            w[4 * k] = v.x;
            w[4 * k + 1] = v.y;
            w[4 * k + 2] = v.z;
            w[4 * k + 3] = v.w;
        } else {
            w[2 * k] = v.x | static_cast<uint64_t>(v.y) << 32;
            w[2 * k + 1] = v.z | static_cast<uint64_t>(v.w) << 32;
        }
    }
    static __device__ __forceinline__ void put_one(Word<T> (&w)[kPairs], int k, Raw v)
    {
        if constexpr (sizeof(Raw) == 2) w[k / 2] |= static_cast<Word<T>>(v) << (16 * (k & 1));
        else w[k / 2] |= static_cast<Word<T>>(__float_as_uint(v)) << (32 * (k & 1));
    }
    __device__ __forceinline__ void store(Raw* row, const Word<T> (&w)[kPairs]) const
    {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if (!has(k)) continue;
            Raw* p = row + (k * lanes + lane) * VEC;
            if constexpr (kChunkBytes == 16) {
                uint4 v;
                if constexpr (sizeof(Word<T>) == 4)
                    v = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                else
                    v = make_uint4(static_cast<uint32_t>(w[2 * k]), static_cast<uint32_t>(w[2 * k] >> 32),
                                   static_cast<uint32_t>(w[2 * k + 1]), static_cast<uint32_t>(w[2 * k + 1] >> 32));
                *reinterpret_cast<uint4*>(p) = v;
            } else if constexpr (VEC == 2) {
                *reinterpret_cast<Word<T>*>(p) = w[k];
            } else if constexpr (sizeof(Raw) == 2) {
                *p = static_cast<Raw>(w[k / 2] >> (16 * (k & 1)));
            } else {
                *p = __uint_as_float(static_cast<uint32_t>(w[k / 2] >> (32 * (k & 1))));
            }
        }
    }
    // Values of a float vector at the thread's columns (`rest` past its end).
    __device__ __forceinline__ void load_f32(uint64_t (&o)[kPairs], const float* v, float rest) const
    {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            float f[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = column(2 * e + q);
                f[q] = c < width ? __ldg(v + c) : rest;
            }
            o[e] = pair(f[0], f[1]);
        }
    }
    // v with zeros past the row.
    __device__ __forceinline__ uint64_t inside(uint64_t v, int e) const
    {
        if constexpr (VEC >= 2) {
            return has(2 * e / VEC) ? v : pair(0.0f, 0.0f);
        } else {
            float lo, hi;
            unpair(lo, hi, v);
            return pair(has(2 * e) ? lo : 0.0f, has(2 * e + 1) ? hi : 0.0f);
        }
    }
};

// Rows ahead of their use, in shared memory, filled by asynchronous copies: a
// ring of kTurns turns of kRows rows (of TENSORS tensors).  Rows whose chunks
// are 16 bytes: each thread copies exactly the bytes that it will read
// itself, so its own wait for its copies is all it needs.  Others (COVER):
// the row's threads copy the aligned 16-byte pieces that cover the row, and a
// barrier comes before its elements are read at their own offset.
template <typename T, int VEC, int CPT, int TENSORS>
struct Ring {
    using S = Slice<T, VEC, CPT>;
    using Raw = typename T::raw;
    static constexpr bool kCover = S::kChunkBytes != 16;
    static constexpr int kThreadBytes = TENSORS * CPT * S::kChunkBytes;  // of one row
    static constexpr int kRows = kThreadBytes <= 64 ? 2 : 1;
    static constexpr int kTurns = kThreadBytes <= 64 ? 2 : kThreadBytes <= 128 ? 3 : 1;
    static constexpr int kSlots = kRows * kTurns;
    static int bytes(int threads, int rows_at_once, int width)
    {
        return kSlots * (kCover ? TENSORS * rows_at_once * cover_bytes(width) : kThreadBytes * threads);
    }
    static __host__ __device__ int cover_bytes(int width)
    {
        return (width * static_cast<int>(sizeof(Raw)) + 15) / 16 * 16 + 16;
    }

    uint8_t* slots;
    int sub;  // COVER: which of the block's rows

    __device__ __forceinline__ uint8_t* own(int slot, int tensor, int k) const
    {
        return slots + (((slot * TENSORS + tensor) * CPT + k) * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) *
                           S::kChunkBytes;
    }
    __device__ __forceinline__ uint8_t* cover(const S& s, int slot, int tensor) const
    {
        return slots + ((sub * kSlots + slot) * TENSORS + tensor) * cover_bytes(s.width);
    }
    // Starts copying the row at `from` (of the tensor that begins at `base`).
    __device__ __forceinline__ void fetch(const S& s, int slot, int tensor, const Raw* base, const Raw* from) const
    {
        if constexpr (!kCover) {
#pragma unroll
            for (int k = 0; k < CPT; ++k)
                if (s.has(k)) {
                    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(own(slot, tensor, k)));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(from + (k * s.lanes + s.lane) * VEC)
                                 : "memory");
                }
        } else {
            uint8_t* to = cover(s, slot, tensor);
            const uintptr_t first = reinterpret_cast<uintptr_t>(from) & ~uintptr_t{15};
            const uintptr_t end = reinterpret_cast<uintptr_t>(from + s.width);
            for (uintptr_t p = first + 16 * s.lane; p < end; p += 16 * s.lanes) {
                uint8_t* dst = to + (p - first);
                if (p >= reinterpret_cast<uintptr_t>(base)) {
                    const int n = end - p < 16 ? static_cast<int>(end - p) : 16;  // no byte past the row
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                                 "l"(p), "r"(n)
                                 : "memory");
                } else {
                    // the tensor begins inside this piece
                    for (const Raw* q = base; q < from + s.width && reinterpret_cast<uintptr_t>(q) < p + 16; ++q)
                        *reinterpret_cast<Raw*>(dst + (reinterpret_cast<uintptr_t>(q) - p)) = __ldg(q);
                }
            }
        }
    }
    __device__ __forceinline__ void read(const S& s, int slot, int tensor, const Raw* from, Word<T> (&w)[S::kPairs]) const
    {
#pragma unroll
        for (int e = 0; e < S::kPairs; ++e) w[e] = 0;
        const uint8_t* row = nullptr;
        if constexpr (kCover) row = cover(s, slot, tensor) + (reinterpret_cast<uintptr_t>(from) & 15);
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
            if constexpr (!kCover) {
                if (s.has(k)) S::put(w, k, *reinterpret_cast<const uint4*>(own(slot, tensor, k)));
            } else {
                // no branch around each element: one past the row reads the last and is dropped
                const int at = k * s.lanes + s.lane, most = (s.width - 1) / VEC;
                if constexpr (VEC == 2) {
                    const Word<T> v = *(reinterpret_cast<const Word<T>*>(row) + min(at, most));
                    w[k] = at <= most ? v : 0;
                } else {
                    const Raw v = *(reinterpret_cast<const Raw*>(row) + min(at, most));
                    S::put_one(w, k, at <= most ? v : Raw(0));
                }
            }
        }
    }
};

__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Moves a ring on by one turn: `fetch(place)` starts the copies of the next
// turn to come into a place of the ring; afterwards the current turn can be read.
template <typename R, bool WARP, typename F>
__device__ __forceinline__ void next_turn(int place, F& fetch)
{
    auto sync = [] {
        if constexpr (WARP) __syncwarp();
        else __syncthreads();
    };
    const int last = place == 0 ? R::kTurns - 1 : place - 1;
    if constexpr (!R::kCover) {
        fetch(last);
        copies_close();
        copies_wait<R::kTurns - 1>();
    } else if constexpr (R::kTurns == 1) {
        sync();
        fetch(0);
        copies_close();
        copies_wait<0>();
        sync();
    } else {
        // others may still read the place that the new copies go to, until the barrier
        copies_wait<R::kTurns - 2>();
        sync();
        fetch(last);
        copies_close();
    }
}

// Sums of N (1, 2 or 4) values over the threads of one row, for all of them.
// Within a warp the values are dealt out over the lanes as they are added:
// N = 4 takes 6 exchanges instead of 20.  Blocks: one barrier a call; `slot`
// alternates between calls, so that no thread overwrites what another still
// reads.
template <bool WARP, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int slot)
{
    const int lane = threadIdx.x & 31;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
    int own = 0;  // which value this lane ends up with
#pragma unroll
    for (int n = N, o = 16; o > 0; o >>= 1) {
        if (n > 1) {
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                const float keep = upper ? x[n / 2 + i] : x[i], give = upper ? x[i] : x[n / 2 + i];
                x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
            n /= 2;
            own = 2 * own + (upper ? 1 : 0);
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
        }
    }
    if constexpr (WARP) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, x[0], i * (32 / N));
    } else {
        float* r = red + slot * 16 * N;
        if ((lane & (32 / N - 1)) == 0) r[16 * own + (threadIdx.x >> 5)] = x[0];
        __syncthreads();
        // Every warp adds the 16 entries of each value (zero past the last
        // warp), 32 / N lanes a value.
        constexpr int kLanes = 32 / N, kEach = kLanes < 16 ? 16 / kLanes : 1;
        float t = r[16 * (lane / kLanes) + (lane % kLanes % 16)];
#pragma unroll
        for (int e = 1; e < kEach; ++e) t += r[16 * (lane / kLanes) + lane % kLanes + e * kLanes];
#pragma unroll
        for (int o = kLanes < 16 ? kLanes / 2 : 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = N == 1 ? t : __shfl_sync(0xffffffffu, t, i * kLanes);
    }
}

__device__ __forceinline__ float sum_of(uint64_t v)
{
    float lo, hi;
    unpair(lo, hi, v);
    return lo + hi;
}

// Threads that the registers must do for: a row takes 512 at most; at 16
// elements a thread the bound of 640 keeps them under 97, for two blocks of
// 320 threads an SM.
template <int ELEMS>
constexpr int kBound = ELEMS == 16 ? 640 : 512;

template <typename S, bool WARP>
__device__ __forceinline__ S make_slice(int width)
{
    return S{WARP ? 32 : static_cast<int>(blockDim.x),
             WARP ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x), width};
}

template <typename T, int VEC, int CPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowsPerBlock : kBound<VEC * CPT>) layer_norm_kernel(const LnArgs a)
{
    using S = Slice<T, VEC, CPT>;
    using R = Ring<T, VEC, CPT, 1>;
    using Raw = typename T::raw;
    constexpr int NP = S::kPairs, NR = R::kRows;
    constexpr bool kHold = NP <= 8;  // weights stay in registers
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ __align__(16) float red[64];
    const S s = make_slice<S, WARP>(a.width);
    const int sub = WARP ? (threadIdx.x >> 5) : 0;
    constexpr int kBlockRows = WARP ? kRowsPerBlock : 1;
    if constexpr (!WARP) {
        for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i] = 0.0f;
        __syncthreads();
    }
    const int64_t g = blockIdx.y;
    const float* w = a.weight ? a.weight + g * a.width : nullptr;
    const float* b = a.bias ? a.bias + g * a.width : nullptr;
    const int step = static_cast<int>(gridDim.x) * kBlockRows;  // from one of the block's rows to its next
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kBlockRows + sub, first = g * a.rows_per_group + r0;
    const int count = r0 < a.rows_per_group ? static_cast<int>((a.rows_per_group - r0 + step - 1) / step) : 0;
    const R ring{dynamic, sub};
    const Raw* x0 = static_cast<const Raw*>(a.x);
    const Raw *to_fetch = x0 + first * a.x_stride, *to_read = to_fetch;
    const int64_t x_step = step * a.x_stride, y_step = step * a.out_stride;
    Raw* y = static_cast<Raw*>(a.out) + first * a.out_stride;
    float2* stats = reinterpret_cast<float2*>(a.stats) + first;
    int fetched = 0;
    auto fetch = [&](int place) {
#pragma unroll
        for (int i = 0; i < NR; ++i, ++fetched, to_fetch += x_step)
            if (fetched < count) ring.fetch(s, place * NR + i, 0, x0, to_fetch);
    };
#pragma unroll
    for (int q = 0; q < R::kTurns - 1; ++q) {
        fetch(q);
        copies_close();
    }
    uint64_t wv[NP], bv[NP];
    const uint64_t zero = pair(0.0f, 0.0f), one = pair(1.0f, 1.0f);
    auto affine = [&]() {
        if (w) s.load_f32(wv, w, 0.0f);
        if (b) s.load_f32(bv, b, 0.0f);
    };
    if constexpr (kHold) {
#pragma unroll
        for (int e = 0; e < NP; ++e) wv[e] = one, bv[e] = zero;
        affine();
    }
    int place = 0;
    for (int done = 0; done < count; done += NR) {
        next_turn<R, WARP>(place, fetch);
        Word<T> x[NR][NP];
        float v[NR], mean[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i, to_read += x_step) {
            ring.read(s, place * NR + i, 0, to_read, x[i]);
            uint64_t t = zero;
#pragma unroll
            for (int e = 0; e < NP; ++e) t = add_pair(t, widen<T>(x[i][e]));
            v[i] = sum_of(t);
        }
        row_sum<WARP>(v, red, 0);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            mean[i] = v[i] * a.inv_width;
            const uint64_t nm = pair(-mean[i], -mean[i]);
            uint64_t t = zero;
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const uint64_t d = s.inside(add_pair(widen<T>(x[i][e]), nm), e);
                t = fma_pair(d, d, t);
            }
            v[i] = sum_of(t);
        }
        row_sum<WARP>(v, red, 1);
        if constexpr (!kHold) affine();
#pragma unroll
        for (int i = 0; i < NR; ++i, y += y_step, stats += step) {
            if (done + i >= count) break;
            const float rstd = rsqrtf(fmaf(v[i], a.inv_width, a.eps));
            const uint64_t nm = pair(-mean[i], -mean[i]), rs = pair(rstd, rstd);
            if (s.lane == 0) *stats = make_float2(mean[i], rstd);
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                uint64_t t = mul_pair(add_pair(widen<T>(x[i][e]), nm), rs);
                if constexpr (kHold) {
                    t = fma_pair(t, wv[e], bv[e]);
                } else {
                    if (w) t = mul_pair(t, wv[e]);
                    if (b) t = add_pair(t, bv[e]);
                }
                x[i][e] = narrow<T>(t);
            }
            s.store(y, x[i]);
        }
        place = place + 1 == R::kTurns ? 0 : place + 1;
    }
    copies_wait<0>();
}

// x and dy are taken from the ring twice, for the sums and, once these are
// known, for dx: that costs less than holding both in registers beside the
// weight gradients.  dx = rstd (g - mean(g) - xh mean(g xh)) is evaluated as
// dy (w rstd) + (x A + B).
template <typename T, int VEC, int CPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kRowsPerBlock : kBound<VEC * CPT>) layer_norm_backward_kernel(const LnArgs a)
{
    using S = Slice<T, VEC, CPT>;
    using R = Ring<T, VEC, CPT, 2>;
    using Raw = typename T::raw;
    constexpr int NP = S::kPairs, NR = R::kRows;
    constexpr bool kHold = NP <= 8;
    extern __shared__ __align__(16) uint8_t dynamic[];  // the ring; then, WARP: [kRowsPerBlock][width] sums
    __shared__ __align__(16) float red[128];
    allow_dependents();
    const S s = make_slice<S, WARP>(a.width);
    const int sub = WARP ? (threadIdx.x >> 5) : 0;
    constexpr int kBlockRows = WARP ? kRowsPerBlock : 1;
    if constexpr (!WARP) {
        for (int i = threadIdx.x; i < 128; i += blockDim.x) red[i] = 0.0f;
        __syncthreads();
    }
    const int64_t g = blockIdx.y;
    const float* w = a.weight ? a.weight + g * a.width : nullptr;
    const int step = static_cast<int>(gridDim.x) * kBlockRows;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kBlockRows + sub, first = g * a.rows_per_group + r0;
    const int count = r0 < a.rows_per_group ? static_cast<int>((a.rows_per_group - r0 + step - 1) / step) : 0;
    const R ring{dynamic, sub};
    const Raw *x0 = static_cast<const Raw*>(a.x), *d0 = static_cast<const Raw*>(a.dy);
    const Raw *x_fetch = x0 + first * a.x_stride, *d_fetch = d0 + first * a.dy_stride;
    const Raw *x_read = x_fetch, *d_read = d_fetch;
    const int64_t x_step = step * a.x_stride, d_step = step * a.dy_stride, o_step = step * a.out_stride;
    Raw* dx = static_cast<Raw*>(a.out) + first * a.out_stride;
    const float2* stats = reinterpret_cast<const float2*>(a.stats) + first;
    int fetched = 0;
    auto fetch = [&](int place) {
#pragma unroll
        for (int i = 0; i < NR; ++i, ++fetched, x_fetch += x_step, d_fetch += d_step)
            if (fetched < count) {
                ring.fetch(s, place * NR + i, 0, x0, x_fetch);
                ring.fetch(s, place * NR + i, 1, d0, d_fetch);
            }
    };
#pragma unroll
    for (int q = 0; q < R::kTurns - 1; ++q) {
        fetch(q);
        copies_close();
    }
    const uint64_t zero = pair(0.0f, 0.0f), one = pair(1.0f, 1.0f);
    uint64_t wv[NP], dw[NP], db[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) wv[e] = one, dw[e] = db[e] = zero;
    if constexpr (kHold) {
        if (w) s.load_f32(wv, w, 0.0f);
    }
    int place = 0, slot = 0;
    for (int done = 0; done < count; done += NR, slot ^= 1) {
        float2 st[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (done + i < count) st[i] = __ldg(stats + i * step);
        next_turn<R, WARP>(place, fetch);
        if constexpr (!kHold) {
            if (w) s.load_f32(wv, w, 0.0f);
        }
        float v[2 * NR];
        // Past the last row the ring holds an old one: not counted.
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            v[2 * i] = v[2 * i + 1] = 0.0f;
            if (done + i >= count) break;
            Word<T> x[NP], dy[NP];
            ring.read(s, place * NR + i, 0, x_read + i * x_step, x);
            ring.read(s, place * NR + i, 1, d_read + i * d_step, dy);
            const uint64_t nm = pair(-st[i].x, -st[i].x), rs = pair(st[i].y, st[i].y);
            uint64_t sg = zero, sgx = zero;
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const uint64_t d = widen<T>(dy[e]);
                const uint64_t t = mul_pair(mul_pair(d, rs), add_pair(widen<T>(x[e]), nm));  // dy xh
                dw[e] = add_pair(dw[e], t);
                db[e] = add_pair(db[e], d);
                sg = fma_pair(d, wv[e], sg);
                sgx = fma_pair(t, wv[e], sgx);
            }
            v[2 * i] = sum_of(sg);
            v[2 * i + 1] = sum_of(sgx);
        }
        row_sum<WARP>(v, red, slot);
#pragma unroll
        for (int i = 0; i < NR; ++i, dx += o_step, stats += step, x_read += x_step, d_read += d_step) {
            if (done + i >= count) break;
            Word<T> x[NP], dy[NP];
            ring.read(s, place * NR + i, 0, x_read, x);
            ring.read(s, place * NR + i, 1, d_read, dy);
            const float mg = v[2 * i] * a.inv_width, mgx = v[2 * i + 1] * a.inv_width;
            const float fa = -st[i].y * st[i].y * mgx, fb = -fmaf(fa, st[i].x, st[i].y * mg);
            const uint64_t ca = pair(fa, fa), cb = pair(fb, fb), rs = pair(st[i].y, st[i].y);
#pragma unroll
            for (int e = 0; e < NP; ++e)
                x[e] = narrow<T>(fma_pair(widen<T>(dy[e]), mul_pair(wv[e], rs), fma_pair(widen<T>(x[e]), ca, cb)));
            s.store(dx, x);
        }
        place = place + 1 == R::kTurns ? 0 : place + 1;
    }
    copies_wait<0>();
    if (!a.partial) return;
    float* part = a.partial + (g * a.parts + blockIdx.x) * 2 * a.width;
    float* merge = reinterpret_cast<float*>(dynamic);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if constexpr (WARP) __syncthreads();
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            float f[2];
            unpair(f[0], f[1], which ? db[e] : dw[e]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = s.column(2 * e + q);
                if (c < a.width) {
                    if constexpr (WARP) merge[sub * a.width + c] = f[q];
                    else part[which * a.width + c] = f[q];
                }
            }
        }
        if constexpr (WARP) {
            // The block's eight warps hold sums of the same columns.
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                float t = 0.0f;
#pragma unroll
                for (int q = 0; q < kRowsPerBlock; ++q) t += merge[q * a.width + c];
                part[which * a.width + c] = t;
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
// else single ones; 16 elements a thread (their weights and both sums of the
// backward pass stay in registers), 32 beyond 8,192 columns, so that a row
// never takes more than 512 threads.
struct Spread {
    int vec, cpt, lanes;
};

Spread spread_of(int esz, int64_t width, bool vec16, bool vec4)
{
    Spread s;
    s.vec = vec16 ? 16 / esz : vec4 && esz == 2 ? 2 : 1;
    const int elems = width <= 256 ? 8 : width <= 8192 ? 16 : 32;
    s.cpt = elems / s.vec;
    s.lanes = static_cast<int>(((width + elems - 1) / elems + 31) / 32 * 32);
    return s;
}

// Blocks along a group's rows, backward: those that are resident at once
// (about 640 threads an SM at 96 registers), fewer where a block would have
// under four rows, for each block adds a partial row to the second kernel's work.
int64_t parts_of(int64_t rows_per_group, int64_t groups, bool warp, int lanes)
{
    const int64_t per_block = warp ? kRowsPerBlock : 4;
    const int64_t want = (rows_per_group + per_block - 1) / per_block;
    const int64_t per_sm = warp ? 2 : (lanes > 320 ? 1 : 640 / lanes);
    int64_t cap = h3qk_internal_sm_count() * per_sm / groups;
    if (cap < 1) cap = 1;
    return want < cap ? want : cap;
}

// The spread a call could use at most parallel (for the size of the workspace,
// which is fixed before alignment is known).
int64_t max_parts(int64_t rows_per_group, int64_t groups)
{
    int64_t cap = h3qk_internal_sm_count() * static_cast<int64_t>(10) / groups;
    if (cap < 1) cap = 1;
    return rows_per_group < cap ? rows_per_group : cap;
}

// Shared memory a block may ask for at launch, beside the kernel's own arrays
// (512 bytes at most): the largest ring is 192 KiB (196,704 bytes).
constexpr int kMostDynamic = 200 * 1024;

// Raises the limit once per kernel and device, whatever this call asks for:
// the default of 48 KiB holds the kernel's own arrays too.
template <typename K>
cudaError_t launch_with(K* kernel, bool (&raised)[64], dim3 grid, int threads, int smem, const LnArgs& a, cudaStream_t st)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!raised[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostDynamic);
        if (e != cudaSuccess) return e;
        raised[dev] = true;
    }
    kernel<<<grid, threads, smem, st>>>(a);
    h3qk_internal_count_launch();
    return cudaGetLastError();
}

template <typename T, int VEC, int CPT, bool WARP>
cudaError_t launch(bool backward, const LnArgs& a, int64_t groups, int lanes, cudaStream_t st)
{
    static bool raised[2][64] = {};
    const int threads = WARP ? 32 * kRowsPerBlock : lanes, rows_at_once = WARP ? kRowsPerBlock : 1;
    if (backward) {
        const dim3 grid(static_cast<unsigned>(a.parts), static_cast<unsigned>(groups));
        const int sums = WARP && a.partial ? kRowsPerBlock * a.width * 4 : 0;
        const int ring = Ring<T, VEC, CPT, 2>::bytes(threads, rows_at_once, a.width);
        return launch_with(layer_norm_backward_kernel<T, VEC, CPT, WARP>, raised[0], grid, threads,
                           sums > ring ? sums : ring, a, st);
    }
    const int64_t want = WARP ? (a.rows_per_group + kRowsPerBlock - 1) / kRowsPerBlock : a.rows_per_group;
    const int64_t per_sm = threads >= 1024 ? 1 : 1024 / threads;
    int64_t cap = h3qk_internal_sm_count() * per_sm / groups;
    if (cap < 1) cap = 1;
    const dim3 grid(static_cast<unsigned>(want < cap ? want : cap), static_cast<unsigned>(groups));
    return launch_with(layer_norm_kernel<T, VEC, CPT, WARP>, raised[1], grid, threads,
                       Ring<T, VEC, CPT, 1>::bytes(threads, rows_at_once, a.width), a, st);
}

// Only the spreads that spread_of can choose are instantiated: 8 elements a
// thread for one warp, 16 for a warp or a block, 32 for a block.
template <typename T, int VEC>
cudaError_t dispatch_vec(bool back, const LnArgs& a, int64_t groups, const Spread& s, cudaStream_t st)
{
    const int elems = s.vec * s.cpt;
    if (elems == 8) return launch<T, VEC, 8 / VEC, true>(back, a, groups, s.lanes, st);
    if (elems == 32) return launch<T, VEC, 32 / VEC, false>(back, a, groups, s.lanes, st);
    if (s.lanes == 32) return launch<T, VEC, 16 / VEC, true>(back, a, groups, s.lanes, st);
    return launch<T, VEC, 16 / VEC, false>(back, a, groups, s.lanes, st);
}

template <typename T, int FULL>
cudaError_t dispatch(bool back, const LnArgs& a, int64_t groups, const Spread& s, cudaStream_t st)
{
    if (s.vec == FULL) return dispatch_vec<T, FULL>(back, a, groups, s, st);
    if constexpr (FULL == 8)
        if (s.vec == 2) return dispatch_vec<T, 2>(back, a, groups, s, st);
    return dispatch_vec<T, 1>(back, a, groups, s, st);
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
