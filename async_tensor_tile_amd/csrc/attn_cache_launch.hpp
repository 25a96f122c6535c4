// attn_cache_launch.hpp -- the definition of launch_attn_cache, for the files
// that instantiate it.
#pragma once

#include "attn_cache.hpp"

namespace att {

constexpr uint32_t kMostGrid = 65535;                                      // a grid's y and z

template <typename T, int FMT, uint32_t DP, uint32_t WAVES>
static void launch_tall(const CacheArgs& a, hipStream_t stream) {
    const uint32_t items = a.blocks * a.parts;
    CacheArgs part = a;
    for (; part.first_item < items; part.first_item += kMostGrid) {
        const uint32_t left = items - part.first_item;
        hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, WAVES>), dim3(a.kv, a.batch, left < kMostGrid ? left : kMostGrid),
                           dim3(64u * WAVES), 0, stream, part);
    }
}

template <typename T, int FMT, uint32_t DP>
static void launch_dim(const CacheArgs& a, hipStream_t stream) {
    if (a.waves == 0) {
        const uint32_t eights = (a.batch * a.blocks * a.parts + 7u) / 8u, y = eights < kMostGrid ? eights : kMostGrid;
        hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, 0>), dim3(8u * a.kv, y, (eights + y - 1u) / y), dim3(kThreads), 0,
                           stream, a);
    } else if constexpr (DP > 128 || (DP == 96 && FMT == KV_SAME)) {
        launch_tall<T, FMT, DP, 4>(a, stream);
    } else if constexpr (FMT != KV_SAME) {
        launch_tall<T, FMT, DP, 8>(a, stream);
    } else {
        if (a.waves == 8) launch_tall<T, FMT, DP, 8>(a, stream);
        else launch_tall<T, FMT, DP, 4>(a, stream);
    }
}

template <typename T, int FMT>
void launch_attn_cache(const CacheArgs& a, hipStream_t stream) {
    switch (padded_dim(a.dim)) {
    case 64: return launch_dim<T, FMT, 64>(a, stream);
    case 96: return launch_dim<T, FMT, 96>(a, stream);
    case 128: return launch_dim<T, FMT, 128>(a, stream);
    case 192: return launch_dim<T, FMT, 192>(a, stream);
    default: return launch_dim<T, FMT, 256>(a, stream);
    }
}

}  // namespace att
