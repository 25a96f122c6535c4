// attn_cache_launch.hpp -- the definition of launch_attn_cache, for the files
// that instantiate it.
#pragma once

#include "attn_cache.hpp"

namespace att {

template <typename T, int FMT, uint32_t DP>
static void launch_dim(const CacheArgs& a, uint32_t groups, hipStream_t stream) {
    if (a.tall) hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, true>), dim3(groups), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, false>), dim3(groups), dim3(kThreads), 0, stream, a);
}

template <typename T, int FMT>
void launch_attn_cache(const CacheArgs& a, uint32_t groups, hipStream_t stream) {
    switch (padded_dim(a.dim)) {
    case 64: return launch_dim<T, FMT, 64>(a, groups, stream);
    case 96: return launch_dim<T, FMT, 96>(a, groups, stream);
    case 128: return launch_dim<T, FMT, 128>(a, groups, stream);
    case 192: return launch_dim<T, FMT, 192>(a, groups, stream);
    default: return launch_dim<T, FMT, 256>(a, groups, stream);
    }
}

}  // namespace att
