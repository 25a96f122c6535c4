// attn_cache_launch.hpp -- the definition of launch_attn_cache, for the files
// that instantiate it.
#pragma once

#include "attn_cache.hpp"

namespace att {

template <typename T, int FMT, uint32_t DP>
static void launch_dim(const CacheArgs& a, hipStream_t stream) {
    constexpr uint32_t most = 65535;                                       // a grid's y and z
    if (!a.tall) {
        const uint32_t eights = (a.batch * a.parts + 7u) / 8u, y = eights < most ? eights : most;
        hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, false>), dim3(8u * a.kv, y, (eights + y - 1u) / y), dim3(kThreads), 0,
                           stream, a);
        return;
    }
    const uint32_t items = a.blocks * a.parts;
    CacheArgs part = a;
    for (; part.first_item < items; part.first_item += most) {
        const uint32_t left = items - part.first_item;
        hipLaunchKernelGGL((k_attn_cache<T, DP, FMT, true>), dim3(a.kv, a.batch, left < most ? left : most),
                           dim3(64u * tall_waves(FMT != KV_SAME, DP)), 0, stream, part);
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
