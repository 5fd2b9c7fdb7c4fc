// Helpers of the attention block's operators (layer norm, the gradient of
// the QK preparation, attention): 16-bit conversions, warp sums, chained
// launches and the host-side checks they share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "h3qk.h"
#include "h3qk_internal.h"

namespace h3qk_ops {

struct F16 { using raw = uint16_t; static constexpr bool kBf16 = false; };
struct BF16 { using raw = uint16_t; static constexpr bool kBf16 = true; };
struct F32 { using raw = float; };

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Chained launches: the first kernel of a pair lets the second be scheduled
// while it still runs; the second waits here before it reads what the first
// wrote.
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename K, typename... A>
cudaError_t launch_chained(K* kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const A&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    h3qk_internal_count_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

inline h3qk_status status_of(cudaError_t e) { return e == cudaSuccess ? H3QK_OK : h3qk_internal_fail_cuda(e); }

}  // namespace h3qk_ops
