// kernel_attn.hip -- attention of a batch behind a shared prefix, over a
// paged cache.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_util.hpp"

namespace att {

constexpr uint32_t kThreads = 256;

struct AttnArgs {
    View q, o, k, v;                 // q, o {dim, heads, q_len, batch}; pools {dim, slots, heads, pages}
    const int32_t* table;
    const int32_t* lens;
    const int32_t* rows;
    uint64_t pitch;
    uint32_t table_rows, row_pages, pages, slots;
    uint32_t prefix_row, prefix_len;
    float scale;
    float* lse;
    uint32_t* err;
};

// One workgroup for one query: a thread for a key, then a thread for an element.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_attn(const AttnArgs a) {
    __shared__ float q[256], p[kThreads], red[kThreads];
    __shared__ int64_t voff[kThreads];
    const uint32_t tid = threadIdx.x, D = (uint32_t)a.q.dim[0];
    const uint32_t h = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
    const uint32_t kvh = h / (uint32_t)(a.q.dim[1] / a.k.dim[2]);
    const uint32_t row = a.rows ? (uint32_t)a.rows[b] : b;
    int64_t own = 0;
    if (row < a.table_rows) {
        own = a.lens[row];
        const int64_t room = (int64_t)a.slots * a.row_pages;
        if (own < 0 || own > room) {
            if (tid == 0) record_page_error(a.err);
            own = own < 0 ? 0 : room;
        }
    } else if (tid == 0) {
        record_page_error(a.err);
    }
    own = own - (int64_t)a.q.dim[2] + 1 + j;
    if (own < 0) own = 0;
    const uint32_t total = a.prefix_len + (uint32_t)own;
    const gbyte* qp = gptr(a.q.base) + h * a.q.stride[1] + j * a.q.stride[2] + b * a.q.stride[3];
    if (tid < D) q[tid] = (float)((const ATT_GLOBAL T*)qp)[tid];
    float top = -INFINITY, sum = 0.0f, acc = 0.0f;
    for (uint32_t base = 0; base < total; base += kThreads) {
        __syncthreads();
        const uint32_t n = base + tid;
        float s = -INFINITY;
        voff[tid] = -1;
        if (n < total) {
            const uint32_t at = n < a.prefix_len ? n : n - a.prefix_len, r = n < a.prefix_len ? a.prefix_row : row;
            const int32_t page = a.table[(uint64_t)r * a.pitch + at / a.slots];
            if ((uint32_t)page < a.pages) {
                const int64_t slot = at % a.slots;
                const ATT_GLOBAL T* kp = (const ATT_GLOBAL T*)(gptr(a.k.base) + page * a.k.stride[3] +
                                                               slot * a.k.stride[1] + kvh * a.k.stride[2]);
                voff[tid] = page * a.v.stride[3] + slot * a.v.stride[1] + kvh * a.v.stride[2];
                s = 0.0f;
                for (uint32_t d = 0; d < D; ++d) s += q[d] * (float)kp[d];
                s *= a.scale;
            } else {
                record_page_error(a.err);
            }
        }
        red[tid] = s;
        __syncthreads();
        for (uint32_t w = kThreads / 2; w; w /= 2) {
            if (tid < w) red[tid] = fmaxf(red[tid], red[tid + w]);
            __syncthreads();
        }
        const float next = fmaxf(top, red[0]), at0 = next == -INFINITY ? 0.0f : next;
        const float fade = expf(top - at0);
        const float e = expf(s - at0);
        p[tid] = e;
        __syncthreads();
        red[tid] = e;
        __syncthreads();
        for (uint32_t w = kThreads / 2; w; w /= 2) {
            if (tid < w) red[tid] += red[tid + w];
            __syncthreads();
        }
        sum = sum * fade + red[0];
        acc *= fade;
        top = next;
        if (tid < D)
            for (uint32_t i = 0; i < kThreads; ++i)
                if (voff[i] >= 0) acc += p[i] * (float)((const ATT_GLOBAL T*)(gptr(a.v.base) + voff[i]))[tid];
    }
    if (tid < D) {
        gbyte* op = gptr(a.o.base) + h * a.o.stride[1] + j * a.o.stride[2] + b * a.o.stride[3];
        ((ATT_GLOBAL T*)op)[tid] = (T)(sum > 0.0f ? acc / sum : 0.0f);
    }
    if (tid == 0 && a.lse)
        a.lse[((uint64_t)b * a.q.dim[2] + j) * a.q.dim[1] + h] = sum > 0.0f ? top + logf(sum) : -INFINITY;
}

static uint64_t workspace(const View&, const View&, uint32_t, uint32_t) { return 16; }

// Shapes of the queries against a pool.
static bool shapes_fit(const View& q, const View& k) {
    return q.dim[0] == k.dim[0] && q.dim[0] % 8 == 0 && q.dim[0] <= 256 && q.dim[1] % k.dim[2] == 0 &&
           q.dim[1] <= 65535 && q.dim[2] <= 65535 && q.dim[3] <= 65535;
}

}  // namespace att

using namespace att;

extern "C" uint64_t attn_workspace(const tmap_t* q, const tmap_t* k_pool, uint32_t prefix_len,
                                   uint32_t suffix_hint) {
    View vq, vk;
    int32_t tq, tk;
    if (view_of(q, 4, &vq, &tq) || view_of(k_pool, 4, &vk, &tk) || !shapes_fit(vq, vk)) return 0;
    return workspace(vq, vk, prefix_len, suffix_hint);
}

extern "C" tmap_status attn_shared_prefix(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool,
                                          const page_table_t* pt, uint32_t prefix_row, uint32_t prefix_len,
                                          const int32_t* d_rows, uint32_t suffix_hint, float scale, const tmap_t* o,
                                          float* d_lse, void* d_ws, uint64_t ws_bytes, void* stream) {
    if (!q || !k_pool || !v_pool || !pt || !o || !d_ws) return TMAP_ERR_NULL;
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    int32_t tq, tk, tv, to;
    tmap_status st = view_of(q, 4, &a.q, &tq);
    if (st == TMAP_OK) st = view_of(k_pool, 4, &a.k, &tk);
    if (st == TMAP_OK) st = view_of(v_pool, 4, &a.v, &tv);
    if (st == TMAP_OK) st = view_of(o, 4, &a.o, &to);
    if (st == TMAP_OK) st = check_table(pt);
    if (st) return st;
    if (!pt->d_lens) return TMAP_ERR_NULL;
    if (tq != TMAP_F16 && tq != TMAP_BF16) return TMAP_ERR_DTYPE;
    if (tk != tq || tv != tq || to != tq || !same_dims(a.q, a.o) || !same_dims(a.k, a.v) || !shapes_fit(a.q, a.k) ||
        (uint64_t)a.k.dim[1] != pt->slots || (uint64_t)a.k.dim[3] != pt->pages || !std::isfinite(scale))
        return TMAP_ERR_UNSUPPORTED;
    if (prefix_len && (prefix_row >= pt->rows || prefix_len > (uint64_t)pt->slots * pt->row_pages))
        return TMAP_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(d_ws) % 16 != 0) return TMAP_ERR_ALIGN;
    if (ws_bytes < workspace(a.q, a.k, prefix_len, suffix_hint)) return TMAP_ERR_UNSUPPORTED;
    a.table = pt->d_table;
    a.lens = pt->d_lens;
    a.rows = d_rows;
    a.pitch = pt->pitch;
    a.table_rows = pt->rows;
    a.row_pages = pt->row_pages;
    a.pages = pt->pages;
    a.slots = pt->slots;
    a.prefix_row = prefix_row;
    a.prefix_len = prefix_len;
    a.scale = scale;
    a.lse = d_lse;
    st = device_error_word(&a.err);
    if (st) return st;
    const dim3 grid((uint32_t)a.q.dim[1], (uint32_t)a.q.dim[2], (uint32_t)a.q.dim[3]);
    if (tq == TMAP_F16) hipLaunchKernelGGL(k_attn<_Float16>, grid, dim3(kThreads), 0, as_stream(stream), a);
    else hipLaunchKernelGGL(k_attn<__bf16>, grid, dim3(kThreads), 0, as_stream(stream), a);
    return check_launch("attn_shared_prefix");
}
