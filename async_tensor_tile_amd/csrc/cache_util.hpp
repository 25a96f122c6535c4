// cache_util.hpp -- what the cache kernels (rotary positions, pages,
// attention) share: views of the public structs, and the device error word.
#pragma once

#include <hip/hip_runtime.h>

#include "att/tile_device.hpp"
#include "host_util.hpp"
#include "kvcache.h"

namespace att {

// A tensor as these kernels see it: base and byte strides, innermost first.
struct View {
    uint64_t base;
    int64_t dim[4];
    int64_t stride[4];      // stride[0] is the element size
};

// A map as a View.  Only plain tiled maps of `rank` dimensions have one.
inline tmap_status view_of(const tmap_t* m, uint32_t rank, View* v, int32_t* dtype) {
    if (!m) return TMAP_ERR_NULL;
    const TmapImpl t = load_map(m);
    if (is_im2col(t)) return TMAP_ERR_UNSUPPORTED;
    if (t.rank != rank) return TMAP_ERR_RANK;
    for (uint32_t d = 0; d < rank; ++d)
        if (t.es[d] != 1) return TMAP_ERR_UNSUPPORTED;
    v->base = t.base;
    for (uint32_t d = 0; d < 4; ++d) {
        v->dim[d] = t.dim[d];
        v->stride[d] = d == 0 ? t.esize : (int64_t)t.stride[d - 1];
    }
    *dtype = t.dtype;
    return TMAP_OK;
}

inline bool same_dims(const View& a, const View& b) {
    for (int d = 0; d < 4; ++d)
        if (a.dim[d] != b.dim[d]) return false;
    return true;
}

// The sizes a page table has to have before any kernel uses it.
inline tmap_status check_table(const page_table_t* pt) {
    if (!pt || !pt->d_table) return TMAP_ERR_NULL;
    if (pt->rows == 0 || pt->rows > 0x7FFFFFFFu || pt->row_pages == 0 || pt->row_pages >= (1u << 21) ||
        pt->pitch < pt->row_pages || pt->pitch >= (1ull << 32) || pt->slots == 0 || pt->pages == 0 || pt->pages > 0x7FFFFFFFu ||
        (uint64_t)pt->slots * pt->row_pages > 0x7FFFFFFFull)
        return TMAP_ERR_UNSUPPORTED;
    return TMAP_OK;
}

// Workgroups along x that one launch holds: HIP counts a grid's threads of one
// dimension in 32 bits.  Calls with more work launch again for the rest.
constexpr uint32_t max_groups(uint32_t threads) { return 0xFFFFFFFFu / threads; }

__device__ __forceinline__ void record_page_error(uint32_t* word) {
    __hip_atomic_fetch_or(word, DEVERR_PAGE, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace att
