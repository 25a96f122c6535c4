// kernel_kv8.hip -- pools of 8-bit codes: their geometry, and tokens read back.
//
// A lane takes 16 codes of a head and its scale, and writes 16 values, two such at
// a time.  Bound by HBM, of whose rate gathered heads of 128 bytes and a line for
// each page's scales reach 84 %: 65536 tokens of 2 x 8 x 128 e4m3 to bf16 (407 MB)
// take 93 us, 4.4 TB/s.  Tokens of a workgroup and items in flight of a lane were
// measured there: 8 and 4 97 us, 16 and 4 99, 4 and 4 93, 2 and 2 99; 8 codes a
// lane, whose stores lie side by side, 115 (twice the address arithmetic); each XCD
// a run of neighbouring tokens 98.
#include <hip/hip_runtime.h>

#include <cstring>

#include "cache_util.hpp"

namespace att {

constexpr uint32_t kReadThreads = 256;
constexpr uint32_t kReadTokens = 4;           // tokens of a workgroup

struct ReadSeg {
    uint64_t src, dst;
    int64_t src_page, src_slot, src_head;     // byte strides
    int64_t dst_head, dst_tok;
};

struct ReadArgs {
    ReadSeg seg[2];
    const int32_t* rows;
    const int32_t* at;
    const int32_t* table;
    uint64_t pitch;
    uint32_t* err;
    uint32_t table_rows, row_pages, pages, slots;
    uint32_t tokens, dim, heads, magic_heads;
    uint32_t e4m3;
};

// Quotient by an invariant below 2^16 of a numerator below 2^24 (0: by 1).
__device__ __forceinline__ uint32_t quotient(uint32_t n, uint32_t d, uint32_t magic) {
    const uint32_t q = fdiv(n, magic);
    return q * d > n ? q - 1u : q;
}

// N codes, four a word, times their scale.
template <uint32_t N>
__device__ __forceinline__ void values_of(const uint32_t (&code)[N / 4], float scale, bool e4m3, float (&y)[N]) {
#pragma unroll
    for (uint32_t w = 0; w < N / 4; ++w) {
        uint32_t c = code[w];
        asm("" : "+v"(c));                    // a whole word, not four loads of a byte
        if (e4m3) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int32_t)c, false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int32_t)c, true);
            y[4 * w] = lo[0] * scale;
            y[4 * w + 1] = lo[1] * scale;
            y[4 * w + 2] = hi[0] * scale;
            y[4 * w + 3] = hi[1] * scale;
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) y[4 * w + i] = (float)(int8_t)(c >> (8u * i)) * scale;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kReadThreads) void k_kv8_read(const ReadArgs a) {
    constexpr uint32_t N = 16;                // codes of an item
    __shared__ int2 where[kReadTokens];       // page (-1: none) and slot
    const uint32_t tid = threadIdx.x, chunks = a.dim / N, step = kReadThreads / chunks;
    const uint32_t x0 = tid / chunks, c = tid - x0 * chunks, items = kReadTokens * 2u * a.heads;
    const uint32_t blocks = (a.tokens - 1u) / kReadTokens + 1u;
    for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const uint32_t t0 = block * kReadTokens;
        if (tid < kReadTokens) {
            int2 w = make_int2(-1, 0);
            if (tid < a.tokens - t0) {
                const int32_t row = a.rows[t0 + tid], at = a.at[t0 + tid];
                if (row >= 0) {
                    const uint32_t col = (uint32_t)at / a.slots;
                    if ((uint32_t)row < a.table_rows && at >= 0 && col < a.row_pages) {
                        const int32_t page = a.table[(uint64_t)(uint32_t)row * a.pitch + col];
                        if ((uint32_t)page < a.pages) w = make_int2(page, (int32_t)((uint32_t)at - col * a.slots));
                    }
                    if (w.x < 0) record_page_error(a.err);
                }
            }
            where[tid] = w;
        }
        __syncthreads();
        constexpr uint32_t U = 2;             // loads in flight per lane
        for (uint32_t i0 = x0; x0 < step && i0 < items; i0 += U * step) {
            uint32_t code[U][N / 4];
            uint16_t scale[U];
            gbyte* dst[U];
#pragma unroll
            for (uint32_t n = 0; n < U; ++n) {
                const uint32_t i = i0 + n * step;
                dst[n] = nullptr;
                if (i >= items) continue;
                const uint32_t y = quotient(i, a.heads, a.magic_heads), h = i - y * a.heads;
                const ReadSeg& g = a.seg[y & 1u];
                const int2 w = where[y / 2u];
                if (w.x < 0) continue;
                const gbyte* p = gptr(g.src) + (int64_t)w.x * g.src_page + (int64_t)h * g.src_head;
                const u32x4 x = *(const ATT_GLOBAL u32x4*)(p + (int64_t)w.y * g.src_slot + c * N);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) code[n][k] = x[k];
                scale[n] = *(const ATT_GLOBAL uint16_t*)(p + scale_offset((uint32_t)w.y, a.slots, a.dim, g.src_slot));
                dst[n] = gptr(g.dst) + (int64_t)(t0 + y / 2u) * g.dst_tok + (int64_t)h * g.dst_head + c * N * sizeof(T);
            }
#pragma unroll
            for (uint32_t n = 0; n < U; ++n) {
                if (!dst[n]) continue;
                float y[N];
                values_of<N>(code[n], __builtin_bit_cast(float, (uint32_t)scale[n] << 16), a.e4m3, y);
                T z[N];
#pragma unroll
                for (uint32_t q = 0; q < N; ++q) z[q] = (T)y[q];
#pragma unroll
                for (uint32_t q = 0; q < sizeof(T); ++q) {
                    u32x4 v;
                    __builtin_memcpy(&v, z + q * (16 / sizeof(T)), 16);
                    __builtin_nontemporal_store(v, (ATT_GLOBAL u32x4*)(dst[n] + q * 16u));
                }
            }
        }
        __syncthreads();                      // the places are read
    }
}

static ReadSeg read_seg(const View& pool, const View& x) {
    return {pool.base, x.base, pool.stride[3], pool.stride[1], pool.stride[2], x.stride[1], x.stride[2]};
}

}  // namespace att

using namespace att;

extern "C" uint32_t kv8_rows(uint32_t slots, uint32_t dim) { return code_rows(slots, dim); }

extern "C" tmap_status kv8_read(int32_t format, const tmap_t* k_pool, const tmap_t* v_pool, const page_table_t* pt,
                                const int32_t* d_rows, const int32_t* d_at, const tmap_t* k, const tmap_t* v,
                                void* stream) {
    if (!k_pool || !v_pool || !pt || !d_rows || !d_at || !k || !v) return TMAP_ERR_NULL;
    ReadArgs a;
    std::memset(&a, 0, sizeof(a));
    View vk, vv, pk, pv;
    int32_t tk, tv, tpk, tpv;
    tmap_status st = view_of(k, 3, &vk, &tk);
    if (st == TMAP_OK) st = view_of(v, 3, &vv, &tv);
    if (st == TMAP_OK) st = view_of(k_pool, 4, &pk, &tpk);
    if (st == TMAP_OK) st = view_of(v_pool, 4, &pv, &tpv);
    if (st == TMAP_OK) st = check_table(pt);
    if (st) return st;
    if (tk != TMAP_F16 && tk != TMAP_BF16 && tk != TMAP_F32) return TMAP_ERR_DTYPE;
    if ((format != KV_INT8 && format != KV_E4M3) || tv != tk || tpk != TMAP_U8 || tpv != TMAP_U8 ||
        !same_dims(vk, vv) || !same_dims(pk, pv) || pk.dim[0] != vk.dim[0] || pk.dim[2] != vk.dim[1] ||
        pk.dim[1] != code_rows(pt->slots, (uint64_t)pk.dim[0]) || pk.dim[3] != pt->pages || vk.dim[1] > 65535 ||
        vk.dim[2] > 0x7FFFFFFF)
        return TMAP_ERR_UNSUPPORTED;
    a.seg[0] = read_seg(pk, vk);
    a.seg[1] = read_seg(pv, vv);
    a.rows = d_rows;
    a.at = d_at;
    a.table = pt->d_table;
    a.pitch = pt->pitch;
    a.table_rows = pt->rows;
    a.row_pages = pt->row_pages;
    a.pages = pt->pages;
    a.slots = pt->slots;
    a.tokens = (uint32_t)vk.dim[2];
    a.dim = (uint32_t)vk.dim[0];
    a.heads = (uint32_t)vk.dim[1];
    a.magic_heads = magic_for(a.heads);
    a.e4m3 = format == KV_E4M3;
    st = device_error_word(&a.err);
    if (st) return st;
    const uint32_t blocks = (a.tokens - 1u) / kReadTokens + 1u;
    const dim3 grid(blocks < max_groups(kReadThreads) ? blocks : max_groups(kReadThreads));
    if (tk == TMAP_F16) hipLaunchKernelGGL(k_kv8_read<_Float16>, grid, dim3(kReadThreads), 0, as_stream(stream), a);
    else if (tk == TMAP_BF16) hipLaunchKernelGGL(k_kv8_read<__bf16>, grid, dim3(kReadThreads), 0, as_stream(stream), a);
    else hipLaunchKernelGGL(k_kv8_read<float>, grid, dim3(kReadThreads), 0, as_stream(stream), a);
    return check_launch("kv8_read");
}
