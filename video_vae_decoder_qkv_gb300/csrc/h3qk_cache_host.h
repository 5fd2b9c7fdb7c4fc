// Host side of the paged cache: what its entry points check alike.
#pragma once

#include "h3qk_cache.cuh"

namespace h3qk_pages {

struct PoolRanges {
    h3qk_detail::Range data[4], lists[2];  // k, v, their scales; table, kv_lens
};

// Checks a cache and describes it to the kernels.  With `written`, no row may
// share memory with another.
H3QK_HIDDEN h3qk_status check_pool(const h3qk_cache* cache, bool written, Pool* pool, PoolRanges* ranges);

}  // namespace h3qk_pages
