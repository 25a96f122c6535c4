// attn_cache.hpp -- the kernels of attention over the paged cache: causal with a sliding
// window and a few first tokens that stay visible, or of a tree of drafted
// tokens; pools of the queries' type or of 8-bit codes.
//
// The rows of a sequence's key / value head are its queries times the heads of
// the group.  A workgroup takes a block of them over the keys that any of them
// sees, as one list: the first tokens, those from the window's reach on, and
// (a tree) the drafted ones, whose tiles stand in descending order so that a
// row's way up its ancestors is walked once.  Few rows (a token a sequence): 32
// in a workgroup, whose waves take tiles of 32 keys in turn.  Many (a prompt):
// 32 a wave, over shared tiles of 64 keys.  Where that leaves the GPU
// unfilled the list is cut into parts, joined by a second launch.
//
// A tile that every row sees whole is not masked.  In the others each lane masks
// the scores of its own row, and infinities and NaN among the values are added
// outside of the product, to the rows that see them.
//
// Codes.  Keys go to the matrix cores as they are (a code is exact in 16 bits)
// and the fp32 scores are multiplied by the keys' scales.  So do values for bf16,
// whose scales multiply the fp32 weights before their rounding.  f16 has no room for
// a weight times any scale: there the power of two in the scale goes to the code and
// the rest of it to the weight.  Either way a weight is rounded once; a value is not,
// but for an f16 code times its power of two that leaves the type's normal numbers:
// an infinity above them, rounded to the steps of the smallest ones below.
//
// What bounds it.  Few rows: HBM.  64 sequences' next tokens, window 8192, 32 heads
// over 8 of 128 elements: bf16 384 us (2.15 GB, 5.6 TB/s), e4m3 230 (1.09 GB, 4.7).
// Many rows: neither the matrix products nor the weights' arithmetic, but how little
// the two overlap.  2048 queries of 32768 tokens: bf16 985 us (1.08 Pflop/s, matrix cores
// busy 51 % of the time, vector units 50 %), e4m3 1145 to 1190 and int8 beside f16 1240 to
// 1290 (36 to 38 %, vector units 53 to 56 %: codes into elements, scales).  With 32 rows a
// wave each product takes an LDS read and a wait of its own.  Short windows: a
// workgroup's start and end, about 15 us, then 2.4 us a tile (5 x 777 queries of int8,
// dim 80: window 1 17 us, 300 30, 600 40).  A few short sequences: the launch and a
// chain of reads, row, length, page, keys: 9.1 us.
// Registers that do not fit go to memory: at dim 128 36 to 68 bytes a lane of the
// kernels for many rows of codes, 28 to 48 of those for few, 12 of the eight waves' in
// 16 bits; at dim 256 116 to 164, 312 for bf16 beside int8; none elsewhere.
#pragma once

#include <hip/hip_runtime.h>

#include "attn_wave.hpp"

namespace att {

constexpr uint32_t kMaxNodes = 1024;

struct CacheArgs {
    View q, o, k, v;                 // q, o {dim, heads, q_len, batch}; pools {dim, slots, heads, pages}
    const int32_t* table;
    const int32_t* lens;
    const int32_t* rows;
    const int32_t* count;
    const int32_t* parent;           // a tree's; else causal
    uint64_t pitch;
    float* lse;
    uint32_t* err;
    f32x4* part_o;
    float2* part_ml;
    uint32_t table_rows, row_pages, pages, slots;
    uint32_t window, sinks;          // window 0: none
    uint32_t dim, q_len, group, kv, batch;
    uint32_t blocks32, blocks;       // of a sequence's key / value head: of 32 rows, of a workgroup's
    uint32_t parts;                  // along the keys
    uint32_t waves;                  // of a workgroup with 32 rows each; 0: few rows, 32 in all
    uint32_t first_item;             // of (block, part) pairs, where a launch does not hold them all
    double per_group, per_slots, per_parts, per_block, per_kv;   // 1 / group, / slots, / parts, / blocks32, / kv
    uint32_t direct;                 // one part: the result is written at once
    float scale;                     // |scale| * log2(e), 1 if that is 0
    uint32_t flip;                   // sign bits to turn in the queries (scale below 0)
    uint32_t zero;                   // the scale is 0
};

typedef __attribute__((address_space(4))) const CacheArgs cargs;
__device__ __forceinline__ cargs& kernel_args() { return *(cargs*)__builtin_amdgcn_kernarg_segment_ptr(); }
// The arguments read again where they are used, not kept in scalar registers.
__device__ __forceinline__ cargs& fresh() {
    cargs* p = &kernel_args();
    asm volatile("" : "+s"(p));
    return *p;
}

// n / d for n, d below 2^31 and per_d = 1 / d: (n + 1/2) / d is at least 2^-32 away
// from a whole number, and the product off by less than 2^-20 of that.
__device__ __forceinline__ uint32_t quotient(uint32_t n, double per_d) { return (uint32_t)(((double)n + 0.5) * per_d); }
// The page of a row that holds a token.
__device__ __forceinline__ uint32_t column_of(cargs& a, uint32_t token) { return quotient(token, a.per_slots); }

// One sequence as the device's arrays say it is.
struct Sequence {
    uint32_t row;        // of the table
    uint32_t len;        // tokens
    uint32_t count;      // queries; 0 where there are none, or something is out of range
};

__device__ __forceinline__ uint32_t asked_of(cargs& a, uint32_t b) {
    return a.count ? (uint32_t)scalar_load(a.count, b) : a.q_len;
}
__device__ __forceinline__ uint32_t count_of(cargs& a, uint32_t asked) { return asked <= a.q_len ? asked : 0u; }

// `record`: what is out of range is recorded.
__device__ __forceinline__ Sequence sequence_of(cargs& a, uint32_t b, bool record) {
    const uint32_t asked = asked_of(a, b);
    Sequence s = {a.rows ? (uint32_t)scalar_load(a.rows, b) : b, 0u, count_of(a, asked)};
    bool bad = asked > a.q_len;
    if (s.count == 0u) {
        if (bad && record && threadIdx.x == 0) record_page_error(a.err);
        return s;
    }
    if (s.row < a.table_rows) {
        const int64_t room = (int64_t)a.slots * a.row_pages, len = scalar_load(a.lens, s.row);
        s.len = (uint32_t)(len < 0 ? 0 : len > room ? room : len);
        bad = s.len != len || (a.parent && s.len < s.count);
    } else {
        bad = true;
    }
    if (bad && record && threadIdx.x == 0) record_page_error(a.err);
    return s;
}

// The keys of a block of rows as one list, i = 0 .. n - 1:
//   [0, few)             tokens 0 ..
//   [few, context)       tokens low .., for causal rows up to the block's last, else up to the drafted ones
//   [drafted, n)         a tree's nodes 0 .. nodes - 1, tile by tile from the last tile to the first
// Indices between and behind these are no keys.
struct Span {
    uint32_t few, low, context, drafted, nodes, tiles, n;
    int32_t first;                   // token of the sequence's first query
    uint32_t all_from, all_to;       // [0, few) and [all_from, all_to) are seen by every row
};

template <uint32_t TILE>
__device__ __forceinline__ Span span_of(cargs& a, const Sequence& s, uint32_t j0, uint32_t j1) {
    Span x = {};
    x.first = (int32_t)s.len - (int32_t)s.count;
    const bool tree = a.parent != nullptr;
    if (tree && x.first < 0) return x;                                   // the nodes are not all there
    const int32_t p0 = tree ? x.first : x.first + (int32_t)j0, p1 = x.first + (int32_t)j1;
    if (!tree && p1 < 0) return x;
    const uint32_t end = tree ? (uint32_t)x.first : (uint32_t)p1 + 1u;   // context tokens
    const uint32_t sinks = a.sinks < end ? a.sinks : end;
    const int64_t reach = (int64_t)p0 - a.window + 1;
    uint32_t from = a.window && reach > 0 ? (uint32_t)reach : 0u;
    from = from < end ? from : end;
    if (from > sinks) {
        x.few = sinks;
        x.low = from;
    }
    x.context = x.few + (end - x.low);
    x.n = x.drafted = x.context;
    if (tree) {
        x.nodes = j1 + 1u;
        x.tiles = (x.nodes + TILE - 1u) / TILE;
        x.drafted = (x.context + TILE - 1u) / TILE * TILE;
        x.n = x.drafted + x.tiles * TILE;
    }
    const int64_t last_reach = (int64_t)p1 - a.window + 1 - x.low;
    x.all_from = x.few + (a.window && last_reach > 0 ? (uint32_t)last_reach : 0u);
    x.all_to = tree ? x.context : p0 < 0 ? 0u : x.few + ((uint32_t)p0 + 1u - x.low);
    return x;
}

// Whether all rows see all of the keys [i, i + TILE).
template <uint32_t TILE>
__device__ __forceinline__ bool seen_by_all(const Span& x, uint32_t i) {
    return i + TILE <= x.all_to && (x.all_from == x.few || i >= x.all_from || i + TILE <= x.few);
}

// The token of key i, -1 where there is none.
template <uint32_t TILE>
__device__ __forceinline__ int32_t token_of(const Span& x, uint32_t i, uint32_t end) {
    if (i >= end) return -1;
    if (i < x.context) return (int32_t)(i < x.few ? i : i - x.few + x.low);
    if (i < x.drafted) return -1;
    const uint32_t u = i - x.drafted, node = (x.tiles - 1u - u / TILE) * TILE + u % TILE;
    return node < x.nodes ? x.first + (int32_t)node : -1;
}

template <uint32_t DP, int FMT>
struct Shared {                       // of many rows
    uint8_t ring[Geo<DP>::ring_bytes];
    uint64_t kaddr[2 * kSegment];     // address of each key's row in the pools
    uint64_t vaddr[2 * kSegment];
    uint64_t there[2 * kSegment / 64];
    float kscale[FMT == KV_SAME ? 4 : 2 * kSegment];
    float vscale[FMT == KV_SAME ? 4 : 2 * kSegment];   // for the weights
    uint16_t vpower[FMT == KV_SAME ? 4 : 2 * kSegment];   // for the codes, as bf16
    uint32_t odd[4];                  // whether a tile's values hold infinities or NaN
    uint16_t parent[kMaxNodes];       // of each node, 0xFFFF: the context
};

constexpr uint32_t kPages = 1024;     // pages of a row that are looked up in LDS

template <uint32_t DP, int FMT>
struct ShortShared {                  // of few rows
    uint8_t ring[Geo<DP>::ring_bytes];
    uint64_t addr[kWaves][2][2 * kOwnTile];   // of a wave's tiles: the keys' rows in the pools, the values'
    float scale[kWaves][2][FMT == KV_SAME ? 4 : 2 * kOwnTile];
    uint16_t vpower[kWaves][2][FMT == KV_SAME ? 4 : kOwnTile];
    int32_t page[kPages];
    uint16_t parent[kMaxNodes];
};

// What a lane's row sees: keys below `few`, keys of [low, high), and of the
// drafted nodes the way up from `node`.
struct Sees {
    uint32_t few, low, high;
    int32_t node;                     // next on the way up, -1: none
    uint32_t steps;                   // from the row's own node to it
    int32_t at;                       // position of the row
};

__device__ __forceinline__ int32_t parent_of(const uint16_t* parent, int32_t node) {
    const uint32_t p = parent[node];
    return p == 0xFFFFu ? -1 : (int32_t)p;
}

__device__ __forceinline__ Sees sees_of(cargs& a, const Span& x, const uint16_t* parent, uint32_t j, bool valid) {
    Sees s = {0u, 0u, 0u, -1, 0u, 0};
    if (!valid || x.n == 0) return s;
    s.at = x.first + (int32_t)j;
    if (a.parent) {
        s.node = (int32_t)j;
        if (a.window) {                                                  // the depth says where the row stands
            int32_t depth = -1;
            for (int32_t up = (int32_t)j; up >= 0; up = parent_of(parent, up)) ++depth;
            s.at = x.first + depth;
        }
    }
    if (s.at < 0) return s;
    const uint32_t end = (uint32_t)s.at + 1u, last = x.context - x.few + x.low;   // tokens, and those of the list
    const int64_t reach = (int64_t)s.at - a.window + 1 - x.low;
    s.few = x.few;
    if (a.window && x.few == 0) s.few = a.sinks < end ? a.sinks : end;
    s.few = s.few < x.context ? s.few : x.context;
    s.low = x.few + (a.window && reach > 0 ? (uint32_t)reach : 0u);
    s.high = x.few + ((end < last ? end : last) - x.low);
    return s;
}

__device__ __forceinline__ uint64_t bits_below(uint32_t x, uint32_t i) {
    return x <= i ? 0ull : x - i >= 64u ? ~0ull : (1ull << (x - i)) - 1ull;
}

// A bit for each of the keys i .. i + TILE - 1 that the lane's row sees.
template <uint32_t TILE>
__device__ __forceinline__ uint64_t seen_bits(cargs& a, const Span& x, Sees& s, const uint16_t* parent, uint32_t i) {
    if (i < x.context || x.tiles == 0)
        return (bits_below(s.high, i) & ~bits_below(s.low, i)) | bits_below(s.few, i);
    if (i >= x.n) return 0;
    const int32_t n0 = (int32_t)((x.tiles - 1u - (i - x.drafted) / TILE) * TILE);
    uint64_t bits = 0;
    while (s.node >= n0) {
        const int32_t in = s.node - n0;
        if (in < (int32_t)TILE &&
            (!a.window || s.steps < a.window || s.at - (int64_t)s.steps < (int64_t)a.sinks))
            bits |= 1ull << in;
        s.node = parent_of(parent, s.node);
        ++s.steps;
    }
    return bits;
}

// Where the keys of the list lie, thread after thread a key: its page first.
template <uint32_t TILE>
__device__ __forceinline__ int32_t page_of_key(cargs& a, const Span& x, uint32_t row, uint32_t i, uint32_t end) {
    const int32_t t = token_of<TILE>(x, i, end);
    if (t < 0) return -1;
    return *(const ATT_GLOBAL int32_t*)(gptr(a.table) + ((uint64_t)row * a.pitch + column_of(a, (uint32_t)t)) * 4u);
}

// Then its addresses, and its scales are asked for.
struct Scales {
    uint16_t k, v;                    // as bf16, 0 where there is no such key
};
template <uint32_t TILE, uint32_t DP, int FMT>
__device__ __forceinline__ Scales place_key(cargs& a, const Span& x, uint32_t head, uint32_t i, uint32_t end,
                                            int32_t page, Shared<DP, FMT>& sh, uint32_t at) {
    const int32_t t = token_of<TILE>(x, i, end);
    const bool ok = t >= 0 && (uint32_t)page < a.pages;
    if (t >= 0 && !ok) record_page_error(a.err);
    const uint32_t slot = (uint32_t)t - column_of(a, (uint32_t)t) * a.slots;
    const uint64_t kh = a.k.base + (uint64_t)(page * a.k.stride[3] + head * a.k.stride[2]);
    const uint64_t vh = a.v.base + (uint64_t)(page * a.v.stride[3] + head * a.v.stride[2]);
    sh.kaddr[at] = ok ? kh + (uint64_t)(slot * a.k.stride[1]) : zero_row();
    sh.vaddr[at] = ok ? vh + (uint64_t)(slot * a.v.stride[1]) : zero_row();
    const uint64_t mask = __ballot(ok);
    if (at % 64u == 0) sh.there[at / 64u] = mask;
    Scales s = {0, 0};
    if (FMT != KV_SAME && ok) {
        s.k = *(const ATT_GLOBAL uint16_t*)(kh + (uint64_t)scale_offset(slot, a.slots, a.dim, a.k.stride[1]));
        s.v = *(const ATT_GLOBAL uint16_t*)(vh + (uint64_t)scale_offset(slot, a.slots, a.dim, a.v.stride[1]));
    }
    return s;
}

__device__ __forceinline__ float scale_value(uint16_t bits) { return __builtin_bit_cast(float, (uint32_t)bits << 16); }

// A scale as the weights' share times the codes' share.  SPLIT: of a normal one the
// codes get the sign and the power of two, the weights 1 .. 2; 0, infinities and NaN
// go to the codes whole.  Else the weights get all of it.
template <bool SPLIT>
__device__ __forceinline__ void split_scale(uint16_t bits, float* weights, uint16_t* codes) {
    const uint32_t power = bits & 0x7F80u;
    const bool normal = power != 0u && power != 0x7F80u;
    *weights = !SPLIT ? scale_value(bits) : normal ? scale_value((uint16_t)((bits & 0x007Fu) | 0x3F80u)) : 1.0f;
    if (SPLIT) *codes = normal ? (uint16_t)(bits & 0xFF80u) : bits;
}

// ---- codes ------------------------------------------------------------------------

// 16 codes as elements: two chunks of 8.  SCALED: times a power of two, which rounds
// only what is below the type's normal numbers, as a 16-bit cache's elements are.
template <typename T, int FMT, bool SCALED>
__device__ __forceinline__ void elements_of(u32x4 code, float scale, typename Vec<T>::v8 (&y)[2]) {
    constexpr bool F16 = std::is_same<T, _Float16>::value;
#pragma unroll
    for (uint32_t w = 0; w < 4; ++w) {
        uint32_t c = code[w];
        asm("" : "+v"(c));                                               // a whole word, not four loads of a byte
        if constexpr (FMT == KV_INT8 && F16 && !SCALED) {
            // 1024 + 128 + c has its bits in place: c with its sign bit turned, below the exponent of 1024
            const uint32_t u = c ^ 0x80808080u;
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                const uint32_t pair = __builtin_amdgcn_perm(0x64646464u, u, i ? 0x04030402u : 0x04010400u);
                const f16x2_t f = __builtin_bit_cast(f16x2_t, pair) - (_Float16)1152.0f;
                y[w / 2u][4u * (w % 2u) + 2u * i] = f[0];
                y[w / 2u][4u * (w % 2u) + 2u * i + 1u] = f[1];
            }
            continue;
        }
        if constexpr (FMT == KV_E4M3 && !SCALED) {                       // exact in both types
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                T* const z = reinterpret_cast<T*>(&y[w / 2u]) + 4u * (w % 2u) + 2u * i;
                if constexpr (F16) {
                    const auto f = i ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true)
                                     : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
                    z[0] = f[0], z[1] = f[1];
                } else {
                    const auto f = i ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true)
                                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
                    z[0] = f[0], z[1] = f[1];
                }
            }
            continue;
        }
        float f[4];
        if (FMT == KV_E4M3) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int32_t)c, false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int32_t)c, true);
            f[0] = lo[0], f[1] = lo[1], f[2] = hi[0], f[3] = hi[1];
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) f[i] = (float)(int8_t)(c >> (8u * i));
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) y[w / 2u][4u * (w % 2u) + i] = (T)(SCALED ? f[i] * scale : f[i]);
    }
}

// A share of a tile of codes: chunks of 16, THREADS apart, from memory to
// registers and, as elements, to the tile's image in LDS.
template <typename T, uint32_t DP, int FMT, uint32_t ROWS, uint32_t THREADS, bool VALUES>
struct CodeCopy {
    static constexpr uint32_t cpr = DP / 16, N = (ROWS * cpr + THREADS - 1u) / THREADS;
    static constexpr bool whole = ROWS * cpr % THREADS == 0;
    u32x4 raw[N];
    __device__ __forceinline__ void load(uint32_t thread, uint32_t dim, const uint64_t* addr) {
        auto each = [&](auto full) {
#pragma unroll
            for (uint32_t n = 0; n < N; ++n) {
                const uint32_t i = n * THREADS + thread, row = i / cpr, c = i - row * cpr;
                if (!whole && i >= ROWS * cpr) break;
                if (decltype(full)::value || c * 16u < dim) raw[n] = *(const ATT_GLOBAL u32x4*)gptr(addr[row] + c * 16u);
                else raw[n] = (u32x4)(0u);
            }
        };
        if (dim == DP) each(std::true_type{});
        else each(std::false_type{});
    }
    // powers: of the rows, for values that take theirs here.
    template <bool SCALED>
    __device__ __forceinline__ void store(uint32_t thread, const uint16_t* powers, uint8_t* tile) const {
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) {
            const uint32_t i = n * THREADS + thread, row = i / cpr, c = i - row * cpr;
            if (!whole && i >= ROWS * cpr) break;
            typename Vec<T>::v8 y[2];
            elements_of<T, FMT, SCALED>(raw[n], SCALED ? scale_value(powers[row]) : 1.0f, y);
            const uint32_t key = VALUES ? Geo<DP>::key_v(row) : Geo<DP>::key_k(row);
            uint8_t* at = tile + row * (DP * 2u);
            *reinterpret_cast<typename Vec<T>::v8*>(at + ((2u * c) ^ key) * 16u) = y[0];
            *reinterpret_cast<typename Vec<T>::v8*>(at + ((2u * c + 1u) ^ key) * 16u) = y[1];
        }
    }
};

// Where the values' scales go.  bf16 holds a weight times any of them: the codes
// go to the product as they are.  f16 does not (a weight of 2^-10 times a scale of
// 2^-17): split.  (2048 queries of 32768 int8 tokens 1240 us; with values that are
// their code times their scale, rounded, 1230, and the result is off by 1.7 times its
// last rounding, not 1.4.  Weights in units of the largest scale: 1277, a token each of
// 64 sequences, window 8192, 258 for 241.)
template <typename T>
constexpr bool kSplitScales = !std::is_same<T, __bf16>::value;

// Weights times their values' scales; a key that the row does not see (MASKED: a
// bit of `sees` each) has no weight, whatever its scale.
template <bool MASKED, uint32_t NB>
__device__ __forceinline__ void scale_weights(f32x16 (&p)[NB], const float* scales, uint64_t sees) {
    const uint32_t hh = lane_id() / 32u;
#pragma unroll
    for (uint32_t n = 0; n < NB; ++n) {
        const uint32_t bits = (uint32_t)(sees >> (32u * n)) >> (4u * hh);
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g) {
            const f32x4 k = *reinterpret_cast<const f32x4*>(scales + 32u * n + 8u * g + 4u * hh);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i)
                p[n][4u * g + i] = !MASKED || bits & (1u << (8u * g + i)) ? p[n][4u * g + i] * k[i] : 0.0f;
        }
    }
}

// Scores times their keys' scales.
template <uint32_t NB>
__device__ __forceinline__ void scale_scores(f32x16 (&s)[NB], const float* scales) {
    const uint32_t hh = lane_id() / 32u;
#pragma unroll
    for (uint32_t n = 0; n < NB; ++n)
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g) {
            const f32x4 k = *reinterpret_cast<const f32x4*>(scales + 32u * n + 8u * g + 4u * hh);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) s[n][4u * g + i] *= k[i];
        }
}

// ---- results ----------------------------------------------------------------------

template <uint32_t DP>
__device__ __forceinline__ f32x4* part_at(cargs& a, uint64_t block) {
    return a.part_o + block * (DP / 8u * 64u);
}
__device__ __forceinline__ uint64_t part_index(cargs& a, uint32_t b, uint32_t head, uint32_t block32, uint32_t part) {
    return (((uint64_t)b * a.kv + head) * a.blocks32 + block32) * a.parts + part;
}

struct Job {
    uint32_t b, head, block, part;
    Sequence seq;
};

// Row r of a sequence's head: query j, and where it and its results lie.
struct Row {
    uint32_t j;
    bool valid;
    const gbyte* q;
    gbyte* o;
    uint64_t lse;
};

__device__ __forceinline__ Row row_of(cargs& a, const Job& job, uint32_t r, uint32_t rows) {
    const uint32_t j = quotient(r, a.per_group), g = r - j * a.group, h = job.head * a.group;
    const gbyte* const q = gptr(a.q.base) + ((int64_t)job.b * a.q.stride[3] + (int64_t)h * a.q.stride[1]);
    gbyte* const o = gptr(a.o.base) + ((int64_t)job.b * a.o.stride[3] + (int64_t)h * a.o.stride[1]);
    return {j, r < rows, q + (j * a.q.stride[2] + g * a.q.stride[1]), o + (j * a.o.stride[2] + g * a.o.stride[1]),
            ((uint64_t)job.b * a.q_len + j) * (a.kv * a.group) + h + g};
}

// Elements d .. d + 3 of a row.
template <typename T>
__device__ __forceinline__ void store_result(const Row& r, uint32_t d, f32x4 x) {
    typename Vec<T>::v4 y;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) y[i] = (T)x[i];
    *(ATT_GLOBAL uint64_t*)(r.o + d * 2u) = __builtin_bit_cast(uint64_t, y);
}

__device__ __forceinline__ void store_lse(cargs& a, const Row& r, float m, float l) {
    a.lse[r.lse] = l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// ---- many rows ----------------------------------------------------------------------

// Waves of 32 rows over shared tiles of 64 keys.  Two stages: while a tile
// is used the next is on its way; a barrier a tile.
template <typename T, uint32_t DP, int FMT, uint32_t WAVES>
__device__ __forceinline__ void tall_part(cargs& a, Shared<DP, FMT>& sh, const Job& job) {
    constexpr uint32_t THREADS = 64u * WAVES, ROWS = 32u * WAVES;
    const uint32_t tid = threadIdx.x, wave = uniform(tid / 64u), lane = lane_id();
    const uint32_t rows = job.seq.count * a.group, first_row = job.block * ROWS;
    const uint32_t last_row = first_row + ROWS < rows ? first_row + ROWS - 1u : rows - 1u;
    const Span x = span_of<kTile>(a, job.seq, uniform(quotient(first_row, a.per_group)),
                                  uniform(quotient(last_row, a.per_group)));
    const uint32_t per = part_keys(x.n, a.parts, kTile);
    const uint32_t k0 = part_begin(x.n, job.part, per), k1 = part_begin(x.n, job.part + 1u, per);
    const uint32_t tiles = (k1 - k0 + kTile - 1u) / kTile;
    const Row row = row_of(a, job, first_row + wave * kRows + lane % 32u, rows);
    const bool busy = first_row + wave * kRows < rows;
    constexpr uint32_t SEG = kSegment / kTile;                            // tiles of a segment
    constexpr uint32_t NG = Geo<DP>::cpr / WAVES;                         // groups a wave copies of a tile's keys
    static_assert(FMT != KV_SAME || Geo<DP>::cpr % WAVES == 0, "every wave copies as many");
    // The threads that place the keys of a segment, one each.
    const bool places = THREADS == kSegment || tid < kSegment;
    constexpr bool CODES = FMT != KV_SAME, SPLIT = CODES && kSplitScales<T>;
    using W = Wave<T, DP, CODES, true>;
    W w;
    w.load_row(a, row.q, row.valid);
    int32_t page = -1;
    Scales scales = {0, 0};
    if (places) {
        page = page_of_key<kTile>(a, x, job.seq.row, k0 + tid, k1);
        scales = place_key<kTile, DP, FMT>(a, x, job.head, k0 + tid, k1, page, sh, tid);
    }
    if (CODES && places) {
        sh.kscale[tid] = scale_value(scales.k);
        split_scale<SPLIT>(scales.v, &sh.vscale[tid], &sh.vpower[tid]);
        page = page_of_key<kTile>(a, x, job.seq.row, k0 + kSegment + tid, k1);
    }
    if (tid < 4u) sh.odd[tid] = 0u;
    __syncthreads();
    Sees sees = sees_of(a, x, sh.parent, row.j, row.valid);
    // Stages of keys first, of values behind them.
    auto keys = [&](uint32_t t) { return sh.ring + (t & 1u) * Geo<DP>::tile_bytes; };
    auto vals = [&](uint32_t t) { return sh.ring + (2u + (t & 1u)) * Geo<DP>::tile_bytes; };
    auto there = [&](uint32_t t) { return uniform64(sh.there[t % (2u * SEG)]); };
    auto in = [&](uint32_t t) { return t % (2u * SEG) * kTile; };         // where a tile's keys are placed
    const uint32_t dim = a.dim;
    auto copy_k = [&](const uint64_t* addr, const uint8_t* to) {
        if (dim == DP) RowCopy<DP, WAVES, false, true>{wave, DP}.template all<NG>(addr, to);
        else RowCopy<DP, WAVES, false>{wave, dim}.template all<NG>(addr, to);
    };
    auto copy_v = [&](const uint64_t* addr, const uint8_t* to) {
        if (dim == DP) RowCopy<DP, WAVES, true, true>{wave, DP}.template all<NG>(addr, to);
        else RowCopy<DP, WAVES, true>{wave, dim}.template all<NG>(addr, to);
    };
    CodeCopy<T, DP, FMT == KV_SAME ? KV_INT8 : FMT, kTile, THREADS, false> kcode;
    CodeCopy<T, DP, FMT == KV_SAME ? KV_INT8 : FMT, kTile, THREADS, true> vcode;
    // What is on its way has arrived, for every wave, and every wave is done
    // with the stages that are filled next.
    auto meet = [&] {
        if (!CODES) wait_vmcnt<0>();
        wait_lgkm0();
        wg_barrier();
    };
    // Addresses of the next segment's keys: pages a step ahead.
    // Codes are asked for a tile earlier, so they are placed a step earlier.
    constexpr uint32_t PLACE = CODES ? 0u : 1u, FETCH = CODES ? SEG - 1u : 0u, AHEAD = CODES ? 2u : 1u;
    auto begin = [&](uint32_t t) {
        meet();
        if (t % SEG == PLACE && places) {
            const uint32_t s = t / SEG + 1u, at = (s & 1u) * kSegment + tid;
            scales = place_key<kTile, DP, FMT>(fresh(), x, job.head, k0 + s * kSegment + tid, k1, page, sh, at);
        }
        if (CODES && t % SEG == 1u && places) {
            const uint32_t at = ((t / SEG + 1u) & 1u) * kSegment + tid;
            sh.kscale[at] = scale_value(scales.k);
            split_scale<SPLIT>(scales.v, &sh.vscale[at], &sh.vpower[at]);
        }
        if (t % SEG == FETCH && places)
            page = page_of_key<kTile>(fresh(), x, job.seq.row, k0 + (t / SEG + AHEAD) * kSegment + tid, k1);
        if (tid == 0) sh.odd[(t + 1u) % 3u] = 0u;
    };
    if (CODES) {
        auto kfirst = kcode, ksecond = kcode;                             // all on their way together
        auto vfirst = vcode;
        kfirst.load(tid, dim, sh.kaddr + in(0));
        vfirst.load(tid, dim, sh.vaddr + in(0));
        ksecond.load(tid, dim, sh.kaddr + in(1));
        kcode.load(tid, dim, sh.kaddr + in(2));
        vcode.load(tid, dim, sh.vaddr + in(1));
        kfirst.template store<false>(tid, nullptr, keys(0));
        vfirst.template store<SPLIT>(tid, sh.vpower + in(0), vals(0));
        ksecond.template store<false>(tid, nullptr, keys(1));
    } else if (tiles) {
        copy_k(sh.kaddr + in(0), keys(0));
        copy_k(sh.kaddr + in(1), keys(1));
        copy_v(sh.vaddr + in(0), vals(0));
    }
    meet();
    // Behind the last tile, keys that are not there are copied and multiplied:
    // two tiles' work at most, and every tile is like the others.
    auto fill = [&](uint32_t t) {
        if (CODES) {
            kcode.template store<false>(tid, nullptr, keys(t));
            vcode.template store<SPLIT>(tid, sh.vpower + in(t + 1u), vals(t + 1u));
            kcode.load(tid, dim, sh.kaddr + in(t + 3u));
            vcode.load(tid, dim, sh.vaddr + in(t + 2u));
        } else {
            copy_k(sh.kaddr + in(t + 2u), keys(t));
            copy_v(sh.vaddr + in(t + 1u), vals(t + 1u));
        }
    };
    const float scale = a.scale;
    f32x16 s[2][2];
    float top = 0.0f;
    uint64_t seen = ~0ull;                                                // of the tile whose scores are at hand, by the lane's row
    // Tile t's scores are there; `known`: so is the largest of them as they are.
    auto finish = [&](uint32_t t, f32x16 (&y)[2], bool known) {
        uint64_t bits = there(t);
        const bool all = seen_by_all<kTile>(x, k0 + t * kTile);
        if (!all) bits &= seen_bits<kTile>(fresh(), x, sees, sh.parent, k0 + t * kTile);
        seen = bits;
        if (!all || bits != ~0ull) w.mask(y, bits);
        if (!all || bits != ~0ull || !known) top = w.largest(scale, y);
    };
    // Infinities and NaN among the values of a tile that some rows do not see
    // whole are added to the rows that see them, and are 0 for the product.
    auto odd_values = [&](uint32_t t, const f32x16 (&p)[2]) {
        uint8_t* const v = vals(t);
        const bool odd = W::template odd_share<false>(v, wave, WAVES, kTile);
        if (odd && lane == 0) sh.odd[t % 3u] = 1u;
        wait_lgkm0();
        wg_barrier();
        if (uniform(sh.odd[t % 3u]) == 0u) return;
        if (busy) w.template add_odd<2>(v, p, seen);
        wait_lgkm0();
        wg_barrier();
        W::template odd_share<true>(v, wave, WAVES, kTile);
        wait_lgkm0();
        wg_barrier();
    };
    auto step = [&](uint32_t t, f32x16 (&y)[2], f32x16 (&next)[2]) {       // a tile that every row sees whole
        begin(t);
        fill(t);
        if (!busy) return;
        top = w.template advance<CODES, CODES, true>(scale, keys(t + 1u), vals(t), top, y, next, sh.kscale + in(t + 1u),
                                                 sh.vscale + in(t));
        finish(t + 1u, next, true);
    };
    if (busy) {
        w.scores(keys(0), s[0]);
        if (CODES) scale_scores(s[0], sh.kscale + in(0));
        finish(0, s[0], false);
    }
    // Tiles of both kinds in loops of their own: in one loop their registers do not
    // fit beside each other.  Above dim 128 those of a tile between two others do not
    // either (2048 queries of 32768 tokens, dim 256: 7570 us, one after the other 4510).
    constexpr bool BETWEEN = DP <= 128;
    for (uint32_t t = 0; t < tiles;) {
        for (; t < tiles && !(BETWEEN && seen_by_all<kTile>(x, k0 + t * kTile)); ++t) {
            begin(t);
            fill(t);
            if (busy) w.weights(scale, s[0]);
            if (CODES && busy) scale_weights<!SPLIT>(s[0], sh.vscale + in(t), seen);
            if ((SPLIT || FMT != KV_INT8) && (BETWEEN || !seen_by_all<kTile>(x, k0 + t * kTile)))
                odd_values(t, s[0]);                                       // an int8 code by itself is a number
            if (!busy) continue;
            typename W::Piece z[2][DP / 32];
            w.read_values(vals(t), 0, z[0]);
            w.values(vals(t), s[0], z);
            w.scores(keys(t + 1u), s[0]);
            if (CODES) scale_scores(s[0], sh.kscale + in(t + 1u));
            finish(t + 1u, s[0], false);
        }
        if constexpr (!BETWEEN) break;
        uint32_t n = 0;
        while (t + n < tiles && seen_by_all<kTile>(x, k0 + (t + n) * kTile)) ++n;
        for (; n > 1u; n -= 2u, t += 2u) {
            step(t, s[0], s[1]);
            step(t + 1u, s[1], s[0]);
        }
        if (n) {
            step(t++, s[0], s[1]);
            s[0][0] = s[1][0];
            s[0][1] = s[1][1];
        }
    }
    wait_vmcnt<0>();                                                       // nothing may land in LDS of a later workgroup
    if (!busy) return;
    cargs& e = fresh();
    const uint32_t hh = lane / 32u;
    const float l = w.total();
    if (e.direct) {
        if (!row.valid) return;
        const Row out = row_of(e, job, first_row + wave * kRows + lane % 32u, rows);
#pragma unroll
        for (uint32_t i = 0; i < DP / 8u; ++i) {
            const uint32_t b = i / 4u, g = i % 4u, d = 8u * i + 4u * hh;
            const f32x4 y = {w.o[b][4u * g], w.o[b][4u * g + 1u], w.o[b][4u * g + 2u], w.o[b][4u * g + 3u]};
            if (d < e.dim) store_result<T>(out, d, l == 0.0f ? (f32x4)(0.0f) : y / l);
        }
        if (lane < 32u && e.lse) store_lse(e, out, w.m, l);
        return;
    }
    const uint64_t at = part_index(e, job.b, job.head, job.block * WAVES + wave, job.part);
    f32x4* out = part_at<DP>(e, at);
#pragma unroll
    for (uint32_t b = 0; b < DP / 32u; ++b)
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g)
            out[(4u * b + g) * 64u + lane] =
                f32x4{w.o[b][4u * g], w.o[b][4u * g + 1u], w.o[b][4u * g + 2u], w.o[b][4u * g + 3u]};
    if (lane < 32u) e.part_ml[at * 32u + lane] = make_float2(w.m, l);
}

// ---- few rows -------------------------------------------------------------------------

// 32 rows: the waves take tiles of 32 keys in turn, each in LDS of its own and
// without a barrier.  A lane works out where one row of a tile lies, a key's or a
// value's, a tile ahead; the pages are looked up in LDS, since the wait for a load
// would be one for the copies in flight too.  Keys are fetched anew while the
// weights are worked out, values while the next scores are.  At the end the waves'
// sums are joined in LDS.
template <typename T, uint32_t DP, int FMT>
__device__ __forceinline__ void short_part(cargs& a, ShortShared<DP, FMT>& sh, const Job& job) {
    const uint32_t tid = threadIdx.x, wave = uniform(tid / 64u), lane = lane_id(), n32 = lane % 32u;
    const uint32_t rows = job.seq.count * a.group, first_row = job.block * kRows;
    const uint32_t last_row = first_row + kRows < rows ? first_row + kRows - 1u : rows - 1u;
    const Span x = span_of<kOwnTile>(a, job.seq, uniform(quotient(first_row, a.per_group)),
                                     uniform(quotient(last_row, a.per_group)));
    const uint32_t per = part_keys(x.n, a.parts, kOwnTile);
    const uint32_t k0 = part_begin(x.n, job.part, per), k1 = part_begin(x.n, job.part + 1u, per);
    const uint32_t tiles = (k1 - k0 + kOwnTile - 1u) / kOwnTile;
    const Row row = row_of(a, job, first_row + n32, rows);
    constexpr uint32_t NP = Geo<DP>::cpr / 2;                             // copies of a tile's keys
    constexpr bool CODES = FMT != KV_SAME, SPLIT = CODES && kSplitScales<T>;
    using W = Wave<T, DP, false, true>;
    // Pages of the list: those of the first tokens, then those from `low` on.
    const uint32_t few_pages = x.few ? column_of(a, x.few - 1u) + 1u : 0u, low_page = column_of(a, x.low);
    auto entry_of = [&](uint32_t column, bool few) { return few ? column : column - low_page + few_pages; };
    auto load_pages = [&](uint32_t p0) {                                  // kPages of them from p0 on
        cargs& e = fresh();
        const ATT_GLOBAL int32_t* const entries = (const ATT_GLOBAL int32_t*)gptr(e.table) + (uint64_t)job.seq.row * e.pitch;
        const uint32_t last = x.n ? entry_of(column_of(e, job.seq.len - 1u), false) : 0u;
#pragma unroll
        for (uint32_t i = 0; i < kPages / kThreads; ++i) {
            const uint32_t p = p0 + i * kThreads + tid;
            if (x.n && p <= last) sh.page[i * kThreads + tid] = entries[p < few_pages ? p : p - few_pages + low_page];
        }
    };
    W w;
    w.load_row(a, row.q, row.valid);
    auto first_page = [&](uint32_t i) {
        const int32_t t = token_of<kOwnTile>(x, i < x.context ? i : x.n - kOwnTile, x.n);   // of the drafted ones the first node
        return t < 0 ? 0u : entry_of(column_of(fresh(), (uint32_t)t), i < x.few);
    };
    uint32_t p0 = first_page(k0);
    load_pages(p0);
    __syncthreads();
    Sees sees = sees_of(a, x, sh.parent, row.j, row.valid);
    uint8_t* const keys = sh.ring + wave * 2u * Geo<DP>::own_bytes;
    uint8_t* const vals = keys + Geo<DP>::own_bytes;
    const float scale = a.scale;
    const uint32_t dim = a.dim, slots = a.slots;
    const uint64_t base = lane < 32u ? a.k.base + (uint64_t)(job.head * a.k.stride[2]) : a.v.base + (uint64_t)(job.head * a.v.stride[2]);
    const uint64_t page_bytes = lane < 32u ? a.k.stride[3] : a.v.stride[3], slot_bytes = lane < 32u ? a.k.stride[1] : a.v.stride[1];
    // Tile t's addresses, and where its keys are there.
    uint64_t scale_at = 0;
    auto place = [&](uint32_t t) -> uint32_t {
        cargs& e = fresh();
        const uint32_t i = k0 + t * kOwnTile + n32;
        const int32_t tok = token_of<kOwnTile>(x, i, k1);
        const uint32_t col = column_of(e, (uint32_t)tok), slot = (uint32_t)tok - col * slots;
        int32_t page = -1;
        if (tok >= 0) {
            const uint32_t p = entry_of(col, i < x.few) - p0;
            page = sh.page[p < kPages ? p : 0u];
            if (p >= kPages) {                                            // many small pages of drafted tokens
                page = *(const ATT_GLOBAL int32_t*)(gptr(e.table) + ((uint64_t)job.seq.row * e.pitch + col) * 4u);
                asm volatile("" : "+v"(page));                            // waited for here
            }
        }
        const bool ok = (uint32_t)page < e.pages && tok >= 0;
        if (tok >= 0 && !ok) record_page_error(e.err);
        const uint64_t at = base + (uint64_t)(uint32_t)page * page_bytes;
        sh.addr[wave][(t / kWaves) & 1u][lane] = ok ? at + (uint64_t)slot * slot_bytes : zero_row();
        scale_at = CODES && ok ? at + (uint64_t)scale_offset(slot, slots, dim, (int64_t)slot_bytes) : 0u;
        return (uint32_t)__ballot(ok);
    };
    // Waited for here: codes asked for behind a scale that is still on its way come
    // later (64 x 1 of 32768 e4m3 tokens, window 8192: 251 us, waited for 229).
    auto own_scale = [&] {
        uint32_t bits = scale_at ? *(const ATT_GLOBAL uint16_t*)scale_at : 0u;
        asm volatile("" : "+v"(bits));
        return (uint16_t)bits;
    };
    CodeCopy<T, DP, FMT == KV_SAME ? KV_INT8 : FMT, kOwnTile, 64, false> kcode;
    CodeCopy<T, DP, FMT == KV_SAME ? KV_INT8 : FMT, kOwnTile, 64, true> vcode;
    auto ask_k = [&](uint32_t t) {
        const uint64_t* addr = sh.addr[wave][(t / kWaves) & 1u];
        if (CODES) kcode.load(lane, dim, addr);
        else if (dim == DP) RowCopy<DP, 1, false, true>{0, DP}.template all<NP>(addr, keys);
        else RowCopy<DP, 1, false>{0, dim}.template all<NP>(addr, keys);
    };
    auto ask_v = [&](uint32_t t) {
        const uint64_t* addr = sh.addr[wave][(t / kWaves) & 1u] + kOwnTile;
        if (CODES) vcode.load(lane, dim, addr);
        else if (dim == DP) RowCopy<DP, 1, true, true>{0, DP}.template all<NP>(addr, vals);
        else RowCopy<DP, 1, true>{0, dim}.template all<NP>(addr, vals);
    };
    // Tiles in runs that one set of pages is enough for: n keys touch n / slots + 3
    // at most (the first, the last, and a cut between the first tokens and the rest).
    const uint64_t enough = (uint64_t)(kPages - 4u) * slots / kOwnTile;
    const uint32_t run = (uint32_t)(enough < (1u << 26) ? enough : 1u << 26) / kWaves * kWaves;
    for (uint32_t t0 = 0; t0 < tiles; t0 += run) {
        if (t0) {
            __syncthreads();                                              // the pages before are used
            p0 = first_page(k0 + t0 * kOwnTile);
            load_pages(p0);
            __syncthreads();
        }
        const uint32_t end = tiles - t0 < run ? tiles : t0 + run;
        uint32_t there = 0;
        uint16_t bits16 = 0;                                              // of the lane's scale
        if (t0 + wave < end) {
            there = place(t0 + wave);
            if (CODES) bits16 = own_scale();
            wait_lgkm0();
            ask_k(t0 + wave);
            ask_v(t0 + wave);
        }
        for (uint32_t t = t0 + wave; t < end; t += kWaves) {
            const uint32_t next = t + kWaves, k = k0 + t * kOwnTile, now = there;
            float* const scales = sh.scale[wave][(t / kWaves) & 1u];
            uint16_t* const powers = sh.vpower[wave][(t / kWaves) & 1u];
            if (CODES) {
                if (lane < kOwnTile) scales[lane] = scale_value(bits16);
                else split_scale<SPLIT>(bits16, &scales[lane], &powers[lane - kOwnTile]);
                wait_lgkm0();
                kcode.template store<false>(lane, nullptr, keys);
                vcode.template store<SPLIT>(lane, powers, vals);
            }
            if (next < end) {
                there = place(next);
                if (CODES) bits16 = own_scale();
            }
            wait_lgkm0();
            if (!CODES) {
                wait_vmcnt<NP>();
            } else if (next < end) {                                      // both as early as can be: most bytes on their way
                ask_k(next);
                ask_v(next);
            }
            f32x16 s[1];
            w.scores(keys, s);
            wait_lgkm0();
            if (!CODES && next < end) ask_k(next);
            if (CODES) scale_scores(s, scales);
            const bool all = seen_by_all<kOwnTile>(x, k);
            uint32_t bits = now;
            if (!all) bits &= (uint32_t)seen_bits<kOwnTile>(fresh(), x, sees, sh.parent, k);
            if (!all || now != ~0u) w.mask(s, bits);
            w.weights(scale, s);
            if (CODES) {
                if (SPLIT || all) scale_weights<false>(s, scales + kOwnTile, bits);
                else scale_weights<true>(s, scales + kOwnTile, bits);
            } else if (next < end) {
                wait_vmcnt<NP>();
            } else {
                wait_vmcnt<0>();
            }
            if ((SPLIT || FMT != KV_INT8) && !all && W::template odd_share<false>(vals, 0, 1, kOwnTile)) {
                w.template add_odd<1>(vals, s, bits);
                wait_lgkm0();
                W::template odd_share<true>(vals, 0, 1, kOwnTile);
                wait_lgkm0();
            }
            typename W::Piece z[2][DP / 32];
            w.read_values(vals, 0, z[0]);
            w.values(vals, s, z);
            wait_lgkm0();
            if (!CODES && next < end) ask_v(next);
        }
    }
    // join the waves
    cargs& e = fresh();
    constexpr uint32_t NF = DP / 8u;
    __syncthreads();
    float2* const ml = reinterpret_cast<float2*>(sh.addr);
    f32x4* const sums = reinterpret_cast<f32x4*>(sh.ring);
    const uint32_t working = tiles < kWaves ? tiles : kWaves;
    const float total = w.total();
    if (lane < 32u) ml[wave * 32u + lane] = make_float2(w.m, total);
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
    for (uint32_t i = 0; i < working; ++i) m = fmaxf(m, ml[i * 32u + n32].x);
    const float at = m == -INFINITY ? 0.0f : m;
    for (uint32_t i = 0; i < working; ++i) l += ml[i * 32u + n32].y * __builtin_amdgcn_exp2f(ml[i * 32u + n32].x - at);
    if (wave < working) {
        const float fade = __builtin_amdgcn_exp2f(w.m - at);
#pragma unroll
        for (uint32_t b = 0; b < DP / 32u; ++b)
#pragma unroll
            for (uint32_t g = 0; g < 4; ++g)
                sums[(wave * NF + 4u * b + g) * 64u + lane] =
                    f32x4{w.o[b][4u * g], w.o[b][4u * g + 1u], w.o[b][4u * g + 2u], w.o[b][4u * g + 3u]} * fade;
    }
    __syncthreads();
    const uint64_t block = part_index(e, job.b, job.head, job.block, job.part);
    f32x4* const out = part_at<DP>(e, block);
    for (uint32_t f = wave; f < NF; f += kWaves) {
        f32x4 y = (f32x4)(0.0f);
        for (uint32_t i = 0; i < working; ++i) y += sums[(i * NF + f) * 64u + lane];
        if (!row.valid) continue;
        const uint32_t d = 8u * f + 4u * (lane / 32u);
        if (!e.direct) out[f * 64u + lane] = y;
        else if (d < e.dim) store_result<T>(row, d, l == 0.0f ? (f32x4)(0.0f) : y / l);
    }
    if (wave == 0 && row.valid && lane < 32u) {
        if (!e.direct) e.part_ml[block * 32u + lane] = make_float2(m, l);
        else if (e.lse) store_lse(e, row, m, l);
    }
}

// WAVES of 32 rows each; 0: few rows, 32 in all, and four waves on them.
template <typename T, uint32_t DP, int FMT, uint32_t WAVES>
__global__ __launch_bounds__(WAVES ? 64 * WAVES : kThreads, DP <= 128 ? 2 : 1) void k_attn_cache(const CacheArgs) {
    constexpr bool TALL = WAVES != 0;
    constexpr uint32_t THREADS = TALL ? 64u * WAVES : kThreads;
    cargs& a = kernel_args();
    __shared__ __attribute__((aligned(1024))) std::conditional_t<TALL, Shared<DP, FMT>, ShortShared<DP, FMT>> sh;
    Job job;
    uint32_t item;
    // Workgroups go to the 8 XCDs in turn, x fastest.
    if constexpr (TALL) {
        // A unit (sequence and head) keeps to few XCDs, to one where the heads are a
        // multiple of 8: its blocks read the same keys (8192 queries of 16384 tokens,
        // window 4096: 593 us, with a block's heads on one XCD 658).  A sequence's
        // last blocks, which see the most, go first.
        item = blockIdx.z + a.first_item;
        job.head = blockIdx.x;
        job.b = blockIdx.y;
    } else {
        // The heads of one (sequence, part) meet in one XCD: where they lie side by
        // side in a token's row, one head alone would keep few of the L2's channels
        // busy.
        item = (blockIdx.z * gridDim.y + blockIdx.y) * 8u + blockIdx.x % 8u;
        job.head = blockIdx.x / 8u;
        if (item >= a.batch * a.blocks * a.parts) return;
    }
    uint32_t rest = a.parts == 1u ? item : uniform(quotient(item, a.per_parts));
    job.part = item - rest * a.parts;
    if constexpr (!TALL) {
        job.b = a.blocks == 1u ? rest : uniform(quotient(rest, a.per_block));   // blocks of 32 rows
        rest -= job.b * a.blocks;
    }
    job.block = a.blocks - 1u - rest;
    job.seq = sequence_of(a, job.b, job.head == 0 && job.part == 0 && job.block == 0);
    if (job.block * (TALL ? THREADS / 2u : kRows) >= job.seq.count * a.group) return;
    if (a.parent) {
        for (uint32_t n = threadIdx.x; n < job.seq.count; n += THREADS) {
            const int32_t p = a.parent[(uint64_t)job.b * a.q_len + n];
            const bool ok = p >= -1 && p < (int32_t)n;
            if (!ok) record_page_error(a.err);
            sh.parent[n] = ok ? (uint16_t)p : (uint16_t)0xFFFFu;
        }
    }
    if constexpr (TALL) tall_part<T, DP, FMT, WAVES>(a, sh, job);
    else short_part<T, DP, FMT>(a, sh, job);
}

// ---- launches (each type and format in a file of its own, so that they build side by side) ----

static inline uint32_t padded_dim(uint32_t dim) {
    return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256;
}

// The products' launch; defined where it is instantiated.
template <typename T, int FMT>
void launch_attn_cache(const CacheArgs& a, hipStream_t stream);

}  // namespace att
