// The instances of the paged tile kernel for fp16 pages, in a unit of
// their own so that they compile in parallel.
#include "h3qk_cache_tiles.cuh"

cudaError_t h3qk_pages::cache_tiles_fp16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st)
{
    return by_shape<false, false>(p, m, grid, st);
}
