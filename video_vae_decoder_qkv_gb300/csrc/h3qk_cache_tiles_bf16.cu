// The instances of the paged tile kernel for bf16 pages, in a unit of
// their own so that they compile in parallel.
#include "h3qk_cache_tiles.cuh"

cudaError_t h3qk_pages::cache_tiles_bf16(const Attn& p, const Maps& m, const TileGrid& grid, cudaStream_t st)
{
    return by_shape<false, true>(p, m, grid, st);
}
