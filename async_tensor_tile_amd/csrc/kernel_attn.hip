// kernel_attn.hip -- attention of a batch behind a shared prefix, over a
// paged cache.
//
// The queries of one key / value head, all sequences and the group's heads
// together, are the rows of one tall product with the prefix: it is read for
// 128 rows at a time.  Each sequence's own tokens are read for its rows alone.
// Both kinds of work are cut along the keys into parts that run in one launch
// (the first is bound by the matrix cores, the second by HBM, and they share
// the compute units); each part leaves the largest score, the sum of weights
// and the weighted sum of values of its rows, and a second launch joins them:
//   m = max_i m_i, w_i = exp(m_i - m), o = sum_i w_i o_i / sum_i w_i l_i.
//
// A wave holds 32 queries.  Scores are computed transposed, keys x queries
// (A = keys from LDS, B = queries in registers), so that a lane owns one query
// and the maximum and the sum over keys stay inside it, up to one exchange
// with the lane 32 further.  The weights, rounded to the element type, then
// already lie as the second product's B operand (values transposed x weights)
// if that product takes its keys in the order 0-3, 8-11 | 4-7, 12-15, which
// the transposing LDS read of the values delivers for free.
//
// Rounding.  Scores, maxima, sums of weights and weighted sums are fp32.  The
// weights alone are rounded, to the element type, since a matrix instruction
// takes both of its sides in one type: against 64 bits the results are then off
// by 0.0023 of their size (root mean square) in bf16 and 0.00027 in f16, where the
// one rounding of the result leaves 0.0017 and 0.00021.  Fp32 weights would take
// a second product of the values with what the rounding left, half as many
// matrix instructions again.
//
// What bounds it.  128 sequences of 32 heads over 8 key / value heads, dim
// 128, behind 32768 shared tokens, up to 1024 own: 122 to 128 us.  The products
// are 70 Gflop (50 us at the 1.4 Pflop/s of a large library product), the keys
// and values 404 MB (78 us at a large copy's 5.2 TB/s; read alone, the own
// tokens take 60 us, 4.5 TB/s).  A tile of the prefix takes a wave 2660 cycles
// at 2.1 GHz, of which its 32 products are 1050 (34 % of the matrix cores' time
// over the launch); the weights' arithmetic costs 380 beside them, the copies
// 550, where the keys lie 170, and the rest is the tile's meeting point and the
// waits between its parts, with one such wave on a SIMD.  Two waves each bring
// the tile to 1600 cycles, at 1.9 GHz, but leave no place for the own tokens'
// loads beside them, and come out slower together.  A few short sequences take
// 11.7 us: two launches, three dependent reads before the first product, the
// join.  Many queries of one sequence are right but not made for: each block of 32
// rows reads all of the sequence's keys, also those behind its last query, and
// masks every tile from the first query's end on (4096 queries, 32 heads over 8,
// no prefix: 0.90 ms).  Above dim 128 the sums and two tiles' scores pass the
// registers: 128 sequences behind 8192 tokens take 42 us at dim 128, 109 at 256.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <type_traits>
#include <utility>

#include "cache_util.hpp"

namespace att {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kRows = 32;                    // queries of a wave
constexpr uint32_t kWgRows = kWaves * kRows;      // queries of a workgroup on the prefix
constexpr uint32_t kTile = 64;                    // keys of a shared tile
constexpr uint32_t kOwnTile = 32;                 // keys of a wave's own tile
constexpr uint32_t kSegment = 256;                // keys whose addresses are worked out together
constexpr float kLazy = 8.0f;                     // powers of two by which a weight may pass 1
constexpr float kLog2e = 1.4426950408889634f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

template <typename T>
struct Vec;
template <>
struct Vec<__bf16> {
    typedef __bf16 v8 __attribute__((ext_vector_type(8)));
    typedef __bf16 v4 __attribute__((ext_vector_type(4)));
    static constexpr uint32_t kExp = 0x7F80u;     // exponent bits: all set for infinities and NaN
};
template <>
struct Vec<_Float16> {
    typedef _Float16 v8 __attribute__((ext_vector_type(8)));
    typedef _Float16 v4 __attribute__((ext_vector_type(4)));
    static constexpr uint32_t kExp = 0x7C00u;
};

__device__ __forceinline__ f32x16 mfma(Vec<__bf16>::v8 a, Vec<__bf16>::v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(Vec<_Float16>::v8 a, Vec<_Float16>::v8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

struct AttnArgs {
    View q, o, k, v;                 // q, o {dim, heads, q_len, batch}; pools {dim, slots, heads, pages}
    const int32_t* table;
    const int32_t* lens;
    const int32_t* rows;
    uint64_t pitch;
    float* lse;
    uint32_t* err;
    f32x4* part_o;                   // partial results: prefix parts, then the sequences' own
    float2* part_ml;
    uint32_t table_rows, row_pages, pages, slots;
    uint32_t prefix_row, prefix_len, hint;
    uint32_t dim, q_len, group, kv;
    uint32_t rows_own, rows_all;     // rows of a key / value head: of one sequence, of all
    uint32_t blocks_all, blocks_own; // the same in blocks of 32
    uint32_t parts_all, parts_own;   // parts along the keys
    uint32_t wg_all, units_all;      // prefix: workgroups; (head, part) pairs
    uint32_t shared;                 // prefix tiles shared by a workgroup's four waves
    uint32_t own_first;              // partial results of the prefix
    uint32_t direct;                 // one part in all: it writes the result
    float scale;                     // |scale| * log2(e), 1 if that is 0
    uint32_t flip;                   // sign bits to turn in the queries (scale below 0)
    uint32_t zero;                   // the scale is 0
};

// The arguments where the launch put them.  A long loop that reads them
// through `fresh` loads them again where it uses them instead of keeping all
// of them in scalar registers, which are too few.
typedef __attribute__((address_space(4))) const AttnArgs cargs;
__device__ __forceinline__ cargs& kernel_args() { return *(cargs*)__builtin_amdgcn_kernarg_segment_ptr(); }
__device__ __forceinline__ cargs& fresh() {
    cargs* p = &kernel_args();
    asm volatile("" : "+s"(p));
    return *p;
}

// A value at an address that is the same for the whole workgroup and that no
// kernel writes meanwhile, through the scalar cache: past the queue of the
// vector loads and copies in flight.
__device__ __forceinline__ int32_t scalar_load(const int32_t* p, uint64_t i) {
    return ((__attribute__((address_space(4))) const int32_t*)(uintptr_t)p)[i];
}

// LDS image of a tile: rows of DP elements (dim rounded up), the 16-byte
// chunks of a row XORed by a key of the row.  64 banks of 4 bytes serve 16
// lanes x 16 bytes or 32 lanes x 8 bytes at once:
//   keys    16 rows at one chunk: the key runs through the chunks of 256 bytes
//           that 16 rows would otherwise share
//   values  4 rows x 4 neighbouring chunks (the transposing read): the key
//           moves groups of 4 chunks
template <uint32_t DP>
struct Geo {
    static constexpr uint32_t cpr = DP / 8;                                   // chunks of a row
    static constexpr uint32_t bits = cpr % 16 == 0 ? 4 : cpr % 8 == 0 ? 3 : 2;
    static constexpr uint32_t period = 16u >> bits;                            // rows that already differ in their banks
    static constexpr uint32_t tile_bytes = kTile * DP * 2;
    static constexpr uint32_t own_bytes = kOwnTile * DP * 2;
    static constexpr uint32_t ring_bytes = 4 * tile_bytes;                     // two stages of keys and values
    static_assert(ring_bytes == kWaves * 2 * own_bytes, "a tile of keys and one of values for each wave");
    static __device__ __forceinline__ uint32_t key_k(uint32_t row) { return (row / period) & ((1u << bits) - 1u); }
    static __device__ __forceinline__ uint32_t key_v(uint32_t row) {
        return bits == 4 ? (row & 3u) << 2 : bits == 3 ? ((row >> 1) & 1u) << 2 : 0u;
    }
};

// One asynchronous 16-byte copy per active lane; the caller waits on vmcnt.
__device__ __forceinline__ void copy16(uint64_t src, uint32_t lds_group) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(lds_group) : "memory");
}

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
    return (uint64_t)uniform((uint32_t)(x >> 32)) << 32 | uniform((uint32_t)x);
}

__device__ __forceinline__ uint32_t part_begin(uint32_t n, uint32_t part, uint32_t per) {
    const uint64_t at = (uint64_t)part * per;
    return at < n ? (uint32_t)at : n;
}
// Keys of one of `parts` parts of n, whole tiles.
__device__ __forceinline__ uint32_t part_keys(uint32_t n, uint32_t parts, uint32_t tile) {
    const uint32_t per = (n + parts - 1u) / parts;
    return (per + tile - 1u) / tile * tile;
}

// The larger, and the sum, of a lane's value and that of the lane 32 further.
struct Halves { float low, high; };
__device__ __forceinline__ Halves halves(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t low = r[0], high = r[1];               // bit_cast of r[1] itself would read r[0]
    return {__builtin_bit_cast(float, low), __builtin_bit_cast(float, high)};
}
__device__ __forceinline__ float max_halves(float x) {
    const Halves h = halves(x);
    return fmaxf(h.low, h.high);
}
__device__ __forceinline__ float add_halves(float x) {
    const Halves h = halves(x);
    return h.low + h.high;
}

// What a key that is not there is read from: keys of 0, whose score is masked,
// and values of 0, so that the weight 0 meets no NaN.  Also the elements of a
// row past dim.
static __device__ __attribute__((aligned(16))) const uint32_t g_zero_row[128] = {};
__device__ __forceinline__ uint64_t zero_row() { return (uint64_t)(uintptr_t)g_zero_row; }

template <uint32_t DP>
struct Shared {
    uint8_t ring[Geo<DP>::ring_bytes];
    uint64_t kaddr[2 * kSegment];     // address of each key's row in the pools
    uint64_t vaddr[2 * kSegment];
    uint64_t there[2 * kSegment / 64];
};

// A wave's 32 queries and what it has summed for them.  Lane l: query l % 32,
// half l / 32 of each group of 8 keys (scores) or 8 elements (result).
template <typename T, uint32_t DP>
struct Wave {
    typedef typename Vec<T>::v8 v8;
    typedef typename Vec<T>::v4 v4;
    static constexpr uint32_t NK = DP / 16, NO = DP / 32;
    v8 q[NK];
    f32x16 o[NO];
    float m, l;                      // largest score seen in powers of two (or below by kLazy at most), sum of weights

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t i = 0; i < NO; ++i) o[i] = (f32x16)(0.0f);
        m = -INFINITY;
        l = 0.0f;
    }

    // Eight elements times 0: infinities and NaN become NaN.
    __device__ __forceinline__ static u32x4 times_zero(u32x4 x) {
        union { u32x4 v; uint16_t e[8]; } y;
        y.v = x;
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) y.e[i] = not_finite(y.e[i]) ? 0x7FFFu : 0u;
        return y.v;
    }

    // The lane's query (row r of the head's rows; none past `rows`).
    __device__ __forceinline__ void load(cargs& a, uint32_t head, uint32_t r, bool valid) {
        const uint32_t lane = lane_id();
        const uint32_t b = r / a.rows_own, in = r - b * a.rows_own, j = in / a.group, g = in - j * a.group;
        const gbyte* p = gptr(a.q.base) + (int64_t)b * a.q.stride[3] + (int64_t)j * a.q.stride[2] +
                         (int64_t)(head * a.group + g) * a.q.stride[1];
#pragma unroll
        for (uint32_t k = 0; k < NK; ++k) {
            const uint32_t d = k * 16u + (lane / 32u) * 8u;
            u32x4 x = (u32x4)(0u);
            if (valid && d < a.dim) x = *(const ATT_GLOBAL u32x4*)(p + d * 2u) ^ a.flip;
            if (a.zero) x = times_zero(x);
            q[k] = __builtin_bit_cast(v8, x);
        }
        clear();
    }

    // Scores of NB blocks of 32 keys.  Keys are read two steps ahead of the
    // product that takes them, no further: the registers are full.
    template <uint32_t NB>
    __device__ __forceinline__ void scores(const uint8_t* keys, f32x16 (&s)[NB]) const {
        constexpr uint32_t AHEAD = 2;
        const uint32_t lane = lane_id(), row = lane % 32u, key = Geo<DP>::key_k(row);
        const uint8_t* at = keys + row * (DP * 2u);
        v8 x[AHEAD + 1][NB];
        auto read = [&](uint32_t k) {
            const uint32_t c = (2u * k + lane / 32u) ^ key;
#pragma unroll
            for (uint32_t n = 0; n < NB; ++n)
                x[k % (AHEAD + 1)][n] = *reinterpret_cast<const v8*>(at + n * 32u * (DP * 2u) + c * 16u);
        };
#pragma unroll
        for (uint32_t k = 0; k < AHEAD; ++k) read(k);
#pragma unroll
        for (uint32_t n = 0; n < NB; ++n) s[n] = (f32x16)(0.0f);
#pragma unroll
        for (uint32_t k = 0; k < NK; ++k) {
            if (k + AHEAD < NK) read(k + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t n = 0; n < NB; ++n) s[n] = mfma(x[k % (AHEAD + 1)][n], q[k], s[n]);
        }
    }

    // Keys that this lane's query does not see, or that are not there (a bit
    // of `sees` each), weigh nothing.
    template <uint32_t NB>
    __device__ __forceinline__ static void mask(f32x16 (&s)[NB], uint64_t sees) {
#pragma unroll
        for (uint32_t n = 0; n < NB; ++n) {
            const uint32_t bits = (uint32_t)(sees >> (32u * n)) >> (4u * (lane_id() / 32u));
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i)
                if (!(bits & (1u << (8u * (i / 4u) + i % 4u)))) s[n][i] = -INFINITY;
        }
    }

    // Largest score of the lane's query, in powers of two.
    template <uint32_t NB>
    __device__ __forceinline__ static float largest(float scale, const f32x16 (&s)[NB]) {
        float top = s[0][0];
#pragma unroll
        for (uint32_t n = 0; n < NB; ++n)
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
        return max_halves(top) * scale;
    }

    // The sums are only rescaled when a score passes the largest of before by
    // 2^kLazy; weights then stay below 2^kLazy, which both types hold.
    // Returns what weights are taken relative to.  Each query goes by its own
    // scores, so its result does not depend on the others of the wave.  A top
    // that is NaN (no score is a number) makes the sums NaN, as it has to.
    __device__ __forceinline__ float rescale(float top) {
        const bool pass = !(top <= m + kLazy);
        if (__any(pass)) {
            const float fade = pass ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
            m = pass ? top : m;
            l *= fade;
#pragma unroll
            for (uint32_t i = 0; i < NO; ++i) o[i] *= fade;
        }
        return m == -INFINITY ? 0.0f : m;
    }

    // Weights of the scores, in place.
    template <uint32_t NB>
    __device__ __forceinline__ void weights(float scale, f32x16 (&s)[NB]) {
        const float at = rescale(largest(scale, s));
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (uint32_t n = 0; n < NB; ++n)
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i) {
                s[n][i] = __builtin_amdgcn_exp2f(fmaf(s[n][i], scale, -at));
                sum[i % 4u] += s[n][i];
            }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    // Values of 16 keys, transposed: NO pieces of 32 elements x 16 keys.
    union Piece { s16x4 h[2]; v8 v; };
    __device__ __forceinline__ static void read_values(const uint8_t* vals, uint32_t step, Piece (&x)[NO]) {
        const uint32_t lane = lane_id(), i = lane % 16u;
        const uint32_t row = 4u * (lane / 32u) + i / 4u;                  // of 4 x 16-element pieces
        const uint32_t c0 = 2u * ((lane / 16u) & 1u) + (i % 4u) / 2u, key = Geo<DP>::key_v(row);
        const uint8_t* at = vals + (step * 16u + row) * (DP * 2u) + 8u * (i & 1u);
#pragma unroll
        for (uint32_t b = 0; b < NO; ++b) {
            const uint8_t* v = at + ((4u * b + c0) ^ key) * 16u;
            x[b].h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v);
            x[b].h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + 8u * DP * 2u));
        }
    }

    // o += values^T x weights; x[0] holds the first step's values.
    template <uint32_t NB>
    __device__ __forceinline__ void values(const uint8_t* vals, const f32x16 (&p)[NB], Piece (&x)[2][NO]) {
#pragma unroll
        for (uint32_t t = 0; t < 2 * NB; ++t) {
            if (t + 1u < 2 * NB) read_values(vals, t + 1u, x[(t + 1u) & 1u]);
            v8 w;
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) w[e] = (T)p[t / 2u][8u * (t & 1u) + e];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t b = 0; b < NO; ++b) o[b] = mfma(x[t & 1u][b].v, w, o[b]);
        }
    }

    // Scores of the next tile of 64 keys, next = keys x q, while this tile's
    // scores become weights, and then o += values^T x weights.  Written as one
    // sequence of matrix instructions with the reads of the ones to come and
    // the arithmetic of the weights spread evenly between them: the matrix
    // cores and the other units work at the same time within a wave.
    // Returns the largest of the next scores.
    __device__ __forceinline__ float advance(float scale, const uint8_t* keys, const uint8_t* vals, float top,
                                             f32x16 (&s)[2], f32x16 (&next)[2]) {
        constexpr uint32_t NS = 2 * NK, NP = 4 * NO, AHEAD = 5;           // products of scores, of values
        const uint32_t lane = lane_id(), row = lane % 32u, key = Geo<DP>::key_k(row);
        const uint8_t* kat = keys + row * (DP * 2u);
        const uint32_t i16 = lane % 16u, vrow = 4u * (lane / 32u) + i16 / 4u;
        const uint32_t c0 = 2u * ((lane / 16u) & 1u) + (i16 % 4u) / 2u, vkey = Geo<DP>::key_v(vrow);
        const uint8_t* vat = vals + vrow * (DP * 2u) + 8u * (i16 & 1u);
        Piece x[AHEAD + 1];
        auto read = [&](uint32_t i) {                                     // what product i takes from LDS
            Piece& y = x[i % (AHEAD + 1u)];
            if (i < NS) {
                const uint32_t k = i / 2u, n = i % 2u;
                y.v = *reinterpret_cast<const v8*>(kat + n * 32u * (DP * 2u) + ((2u * k + lane / 32u) ^ key) * 16u);
            } else if (i < NS + NP) {
                const uint32_t t = (i - NS) / NO, b = (i - NS) % NO;
                const uint8_t* v = vat + t * 16u * (DP * 2u) + ((4u * b + c0) ^ vkey) * 16u;
                y.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)v);
                y.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(v + 8u * DP * 2u));
            }
        };
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) read(i);
        const float at = rescale(top);
        float sum[2] = {0.0f, 0.0f};
        v8 w[4];
        float best = 0.0f;
        static_for<(int)(NS + NP)>([&](auto slot) {
            constexpr uint32_t i = decltype(slot)::value;
            read(i + AHEAD);
            const v8 y = x[i % (AHEAD + 1u)].v;
            if constexpr (i < NS) {
                constexpr uint32_t k = i / 2u, n = i % 2u;
                next[n] = mfma(y, q[k], k == 0 ? (f32x16)(0.0f) : next[n]);
            } else {
                constexpr uint32_t t = (i - NS) / NO, b = (i - NS) % NO;
                o[b] = mfma(y, w[t], o[b]);
            }
            // weight e before product NS + NO * (e / 8) takes it
            constexpr uint32_t M = NS + 3u * NO, e0 = (i * 32u + M - 1u) / M, e1 = ((i + 1u) * 32u + M - 1u) / M;
            static_for<(int)(i < M ? e1 - e0 : 0u)>([&](auto which) {
                constexpr uint32_t e = e0 + decltype(which)::value;
                static_assert(e < 32u && (i < NS || e / 8u > (i - NS) / NO), "in time");
                const float p = __builtin_amdgcn_exp2f(fmaf(s[e / 16u][e % 16u], scale, -at));
                sum[e % 2u] += p;
                asm volatile("" : "+v"(sum[e % 2u]));                     // here, not behind the last product
                w[e / 8u][e % 8u] = (T)p;
            });
            // the next scores' largest, from the third product of values on
            constexpr uint32_t per = (32u + NP - 3u) / (NP - 2u), j0 = i < NS + 2u ? 32u : (i - NS - 2u) * per;
            static_for<(int)(j0 < 32u ? (32u - j0 < per ? 32u - j0 : per) : 0u)>([&](auto which) {
                constexpr uint32_t j = j0 + decltype(which)::value;
                if constexpr (j == 0) best = next[0][0];
                else best = fmaxf(best, next[j / 16u][j % 16u]);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
        l += sum[0] + sum[1];
        return max_halves(best) * scale;
    }

    // Whether a tile of 32 keys holds infinities or NaN in the values of keys
    // [from, to), and those elements become 0.
    __device__ __forceinline__ static bool not_finite(uint16_t x) { return (x & Vec<T>::kExp) == Vec<T>::kExp; }
    template <bool CLEAR>
    __device__ __forceinline__ static bool odd_values(uint8_t* vals, uint32_t from, uint32_t to) {
        bool odd = false;
        for (uint32_t i = lane_id(); i < kOwnTile * Geo<DP>::cpr; i += 64u) {
            const uint32_t row = i / Geo<DP>::cpr;
            if (row < from || row >= to) continue;
            union { u32x4 v; uint16_t e[8]; } x;
            x.v = *reinterpret_cast<const u32x4*>(vals + i * 16u);
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e)
                if (not_finite(x.e[e])) {
                    odd = true;
                    x.e[e] = 0;
                }
            if (CLEAR) *reinterpret_cast<u32x4*>(vals + i * 16u) = x.v;
        }
        return __any(odd);
    }

    // Keys that some queries of the wave see and others do not: an infinity or
    // a NaN among their values must not meet the weight 0 of the latter.  Such
    // elements are added here to the queries that see them, and are 0 for the
    // matrix product.
    __device__ __forceinline__ void ragged_values(uint8_t* vals, const f32x16 (&p)[1], uint32_t limit, uint32_t from,
                                                  uint32_t to) {
        if (!odd_values<false>(vals, from, to)) return;
        const uint32_t hh = lane_id() / 32u;
        for (uint32_t key = from; key < to; ++key) {
            const uint32_t at = 4u * (key / 8u) + key % 4u;
            float x = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < 16; ++i)
                if (i == at && (key >> 2 & 1u) == hh) x = p[0][i];
            x = (float)(T)add_halves(x);
            const uint8_t* row = vals + key * (DP * 2u) + 8u * hh;
#pragma unroll
            for (uint32_t f = 0; f < DP / 8u; ++f) {
                const uint64_t bits = *reinterpret_cast<const uint64_t*>(row + (f ^ Geo<DP>::key_v(key)) * 16u);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const uint16_t h = (uint16_t)(bits >> (16u * e));
                    if (not_finite(h) && key < limit)
                        o[f / 4u][4u * (f % 4u) + e] += x * (float)__builtin_bit_cast(T, h);
                }
            }
        }
        odd_values<true>(vals, from, to);
    }

    // Sum of the weights over both halves.
    __device__ __forceinline__ float total() const { return add_halves(l); }
};

// Where the keys of a row lie, thread after thread a key: first its page, then
// its addresses; what is not a page of the pool is recorded and left out.
// The division by the page's slots is the compiler's: by a multiplication with
// a reciprocal from the host, 128 sequences behind 32768 keys took 136.6 us
// against 135.4.
__device__ __forceinline__ int32_t page_of_key(cargs& a, uint32_t row, uint32_t key, uint32_t end) {
    if (key >= end) return -1;
    return *(const ATT_GLOBAL int32_t*)(gptr(a.table) + ((uint64_t)row * a.pitch + key / a.slots) * 4u);
}

template <uint32_t DP>
__device__ __forceinline__ void place_key(cargs& a, uint32_t head, uint32_t key, uint32_t end, int32_t page,
                                          Shared<DP>& sh, uint32_t at) {
    const bool ok = key < end && (uint32_t)page < a.pages;
    if (key < end && !ok) record_page_error(a.err);
    const int64_t slot = key % a.slots;
    sh.kaddr[at] = ok ? a.k.base + (uint64_t)(page * a.k.stride[3] + slot * a.k.stride[1] + head * a.k.stride[2]) : zero_row();
    sh.vaddr[at] = ok ? a.v.base + (uint64_t)(page * a.v.stride[3] + slot * a.v.stride[1] + head * a.v.stride[2]) : zero_row();
    const uint64_t mask = __ballot(ok);
    if (at % 64u == 0) sh.there[at / 64u] = mask;
}

// Copy n of N of a wave's share of a tile: groups first, first + STEP, ... of
// 64 chunks each.  Chunk i = 64 * group + lane is row i / cpr; the row's
// address says where it lies.
template <uint32_t DP, uint32_t STEP, bool VALUES>
struct RowCopy {
    uint32_t first, dim;
    // Rows from one of the wave's groups to the next; where that is a whole
    // number of periods of the rows' key, a lane's chunk is the same in all.
    static constexpr uint32_t rows = STEP * 64u / Geo<DP>::cpr;
    static constexpr bool same = STEP * 64u % Geo<DP>::cpr == 0 && rows % (VALUES ? 4u : 16u) == 0;
    __device__ __forceinline__ uint32_t chunk(uint32_t n, uint32_t& row) const {
        const uint32_t i = (first + (same ? 0u : n * STEP)) * 64u + lane_id(), r = i / Geo<DP>::cpr;
        row = r + (same ? n * rows : 0u);
        return (i - r * Geo<DP>::cpr) ^ (VALUES ? Geo<DP>::key_v(r) : Geo<DP>::key_k(r));
    }
    __device__ __forceinline__ uint64_t source(uint32_t n, const uint64_t* addr) const {
        uint32_t row;
        const uint32_t c = chunk(n, row);
        const uint64_t at = addr[row] + c * 16u;
        const uint64_t in = (uint64_t)((int64_t)(int32_t)(c * 8u - dim) >> 32);   // all ones below dim, without a branch
        return (at & in) | (zero_row() & ~in);
    }
    __device__ __forceinline__ void issue(uint32_t n, uint64_t src, uint32_t lds) const {
        copy16(src, lds + (first + n * STEP) * 1024u);
    }
    template <uint32_t N>
    __device__ __forceinline__ void all(const uint64_t* addr, const uint8_t* dst) const {
        const uint32_t lds = uniform(lds_addr_of(dst));
        uint64_t src[N];
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) src[n] = source(n, addr);
#pragma unroll
        for (uint32_t n = 0; n < N; ++n) issue(n, src[n], lds);
    }
};

// ---- partial results -------------------------------------------------------------

// A block of 32 rows leaves its (m, l) by row and its sums as the lanes hold
// them: piece f = 4 * b + g of lane l is elements 32 b + 8 g + 4 (l / 32) + 0..3
// of row l % 32.
template <uint32_t DP>
__device__ __forceinline__ f32x4* part_at(cargs& a, uint64_t block) {
    return a.part_o + block * (DP / 8u * 64u);
}

template <typename T>
__device__ __forceinline__ void store_result(cargs& a, uint32_t head, uint32_t r, uint32_t d, f32x4 x) {
    const uint32_t b = r / a.rows_own, in = r - b * a.rows_own, j = in / a.group, g = in - j * a.group;
    gbyte* p = gptr(a.o.base) + (int64_t)b * a.o.stride[3] + (int64_t)j * a.o.stride[2] +
               (int64_t)(head * a.group + g) * a.o.stride[1];
    typename Vec<T>::v4 y;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) y[i] = (T)x[i];
    *(ATT_GLOBAL uint64_t*)(p + d * 2u) = __builtin_bit_cast(uint64_t, y);
}

__device__ __forceinline__ void store_lse(cargs& a, uint32_t head, uint32_t r, float m, float l) {
    const uint32_t b = r / a.rows_own, in = r - b * a.rows_own, j = in / a.group, g = in - j * a.group;
    a.lse[((uint64_t)b * a.q_len + j) * ((uint64_t)a.kv * a.group) + head * a.group + g] =
        l == 0.0f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// ---- the prefix, shared -----------------------------------------------------------

// Four waves of 32 rows each over the tiles of one part of the prefix.  Two
// stages: while a tile is used the next is on its way; a barrier a tile.
template <typename T, uint32_t DP>
__device__ __forceinline__ void shared_part(cargs& a, Shared<DP>& sh, uint32_t head, uint32_t part,
                                            uint32_t block) {
    const uint32_t tid = threadIdx.x, wave = uniform(tid / 64u);
    const uint32_t per = part_keys(a.prefix_len, a.parts_all, kTile);
    const uint32_t k0 = part_begin(a.prefix_len, part, per), k1 = part_begin(a.prefix_len, part + 1u, per);
    const uint32_t tiles = (k1 - k0 + kTile - 1u) / kTile;
    const uint32_t r = block * kWgRows + wave * kRows + lane_id() % 32u;
    constexpr uint32_t SEG = kSegment / kTile;                            // tiles of a segment
    constexpr uint32_t NG = Geo<DP>::cpr / kWaves;                        // groups a wave copies of a tile's keys
    Wave<T, DP> w;
    w.load(a, head, r, r < a.rows_all);
    int32_t page = page_of_key(a, a.prefix_row, k0 + tid, k1);
    place_key(a, head, k0 + tid, k1, page, sh, tid);
    __syncthreads();
    // Stages of keys first, of values behind them.
    auto keys = [&](uint32_t t) { return sh.ring + (t & 1u) * Geo<DP>::tile_bytes; };
    auto vals = [&](uint32_t t) { return sh.ring + (2u + (t & 1u)) * Geo<DP>::tile_bytes; };
    auto there = [&](uint32_t t) { return uniform64(sh.there[t % (2u * SEG)]); };
    const RowCopy<DP, kWaves, false> kcopy{wave, a.dim};
    const RowCopy<DP, kWaves, true> vcopy{wave, a.dim};
    auto kaddr = [&](uint32_t t) { return sh.kaddr + t % (2u * SEG) * kTile; };
    auto vaddr = [&](uint32_t t) { return sh.vaddr + t % (2u * SEG) * kTile; };
    // What is on its way has arrived, for every wave, and every wave is done
    // with the stages that are filled next.
    auto meet = [&] {
        wait_vmcnt<0>();
        wait_lgkm0();
        wg_barrier();
    };
    auto begin = [&](uint32_t t) {
        meet();
        const uint32_t next = k0 + (t / SEG + 1u) * kSegment + tid;
        if (t % SEG == 1)                                                  // used from the next segment's first keys on
            place_key(fresh(), head, next, k1, page, sh, ((t / SEG + 1u) & 1u) * kSegment + tid);
        if (t % SEG == 0) page = page_of_key(fresh(), fresh().prefix_row, next, k1);
    };
    if (tiles) {
        kcopy.template all<NG>(kaddr(0), keys(0));
        kcopy.template all<NG>(kaddr(1), keys(1));
        vcopy.template all<NG>(vaddr(0), vals(0));
    }
    meet();
    if (block * kWgRows + wave * kRows >= a.rows_all) {                    // no rows for this wave: it only copies
        for (uint32_t t = 0; t < tiles; ++t) {
            begin(t);
            kcopy.template all<NG>(kaddr(t + 2u), keys(t));
            vcopy.template all<NG>(vaddr(t + 1u), vals(t + 1u));
        }
        wait_vmcnt<0>();
        return;
    }
    const float scale = a.scale;
    f32x16 s[2][2];
    w.scores(keys(0), s[0]);
    float top = 0.0f;
    auto finish = [&](uint32_t t, f32x16 (&x)[2], bool known) {            // tile t's scores are there
        const uint64_t sees = there(t);
        if (sees != ~0ull) w.mask(x, sees);
        if (sees != ~0ull || !known) top = w.largest(scale, x);
    };
    finish(0, s[0], false);
    // Behind the last tile, keys that are not there are copied and multiplied:
    // two tiles' work at most, and every tile is like the others.
    auto step = [&](uint32_t t, f32x16 (&x)[2], f32x16 (&y)[2]) {
        begin(t);
        kcopy.template all<NG>(kaddr(t + 2u), keys(t));
        vcopy.template all<NG>(vaddr(t + 1u), vals(t + 1u));
        top = w.advance(scale, keys(t + 1u), vals(t), top, x, y);
        finish(t + 1u, y, true);
    };
    for (uint32_t t = 0; t < tiles; ++t) {
        step(t, s[0], s[1]);
        if (++t == tiles) break;
        step(t, s[1], s[0]);
    }
    wait_vmcnt<0>();                                                       // nothing may land in LDS of a later workgroup
    cargs& e = fresh();
    const uint32_t lane = lane_id();
    const uint64_t at = ((uint64_t)head * e.parts_all + part) * e.blocks_all + block * kWaves + wave;
    f32x4* out = part_at<DP>(e, at);
#pragma unroll
    for (uint32_t b = 0; b < DP / 32u; ++b)
#pragma unroll
        for (uint32_t g = 0; g < 4; ++g)
            out[(4u * b + g) * 64u + lane] =
                f32x4{w.o[b][4u * g], w.o[b][4u * g + 1u], w.o[b][4u * g + 2u], w.o[b][4u * g + 3u]};
    const float l = w.total();
    if (lane < 32u) e.part_ml[at * 32u + lane] = make_float2(w.m, l);
}

// ---- a wave's own tiles -------------------------------------------------------------

// 32 rows (of one sequence, or of a prefix with few) over keys [k0, k1) of a
// table row: the waves take tiles of 32 keys in turn, each in LDS of its own,
// so that no barrier is needed: keys are fetched anew while the weights are
// worked out, values while the next scores are.  At the end the waves' sums
// are joined in LDS.
struct OwnJob {
    uint32_t head, row, k0, k1;      // keys [k0, k1) of a table row
    uint32_t first, count;           // rows of the head
    int64_t len;                     // tokens of the sequence; its query j sees len - q_len + 1 + j of them
    bool all;                        // every query sees every key
    uint64_t block;                  // of the partial results
};

template <typename T, uint32_t DP>
__device__ __forceinline__ void own_part(cargs& a, Shared<DP>& sh, const OwnJob& job) {
    const uint32_t tid = threadIdx.x, wave = uniform(tid / 64u), lane = lane_id(), n32 = lane % 32u;
    const uint32_t r = job.first + n32;
    const bool valid = n32 < job.count;
    constexpr uint32_t NP = Geo<DP>::cpr / 2;                             // copies of a tile's keys
    constexpr uint32_t SEG = 2 * kSegment;
    int32_t page[SEG / kThreads];                                         // of the next segment's keys
    auto pages = [&](uint32_t base) {
        cargs& e = fresh();
#pragma unroll
        for (uint32_t i = 0; i < SEG / kThreads; ++i)
            page[i] = page_of_key(e, job.row, base + i * kThreads + tid, job.k1);
    };
    pages(job.k0);                                                        // on its way while the queries are
    Wave<T, DP> w;
    w.load(a, job.head, r, valid);
    // keys below `common` are seen by all of the rows, those below `limit` by this lane's
    const int64_t first_sees = job.len - a.q_len + 1;
    const uint32_t common = job.all ? job.k1 : first_sees < 0 ? 0u : (uint32_t)first_sees;
    const int64_t sees = job.all ? (int64_t)job.k1 : first_sees + (r % a.rows_own) / a.group;
    uint8_t* const keys = sh.ring + wave * 2u * Geo<DP>::own_bytes;
    uint8_t* const vals = keys + Geo<DP>::own_bytes;
    const float scale = a.scale;
    const uint32_t q_len = a.q_len;
    const RowCopy<DP, 1, false> kcopy{0, a.dim};
    const RowCopy<DP, 1, true> vcopy{0, a.dim};
    for (uint32_t base = job.k0; base < job.k1; base += SEG) {
        if (base != job.k0) __syncthreads();                              // the segment before is used up
#pragma unroll
        for (uint32_t i = 0; i < SEG / kThreads; ++i)
            place_key(a, job.head, base + i * kThreads + tid, job.k1, page[i], sh, i * kThreads + tid);
        __syncthreads();
        pages(base + SEG);
        const uint32_t left = job.k1 - base, n = left < SEG ? left : SEG, tiles = (n + kOwnTile - 1u) / kOwnTile;
        auto mask_of = [&](uint32_t t) { return (uint32_t)(uniform64(sh.there[t / 2u]) >> (32u * (t & 1u))); };
        auto issue_k = [&](uint32_t t) { kcopy.template all<NP>(sh.kaddr + t * kOwnTile, keys); };
        auto issue_v = [&](uint32_t t) { vcopy.template all<NP>(sh.vaddr + t * kOwnTile, vals); };
        if (wave < tiles) {
            issue_k(wave);
            issue_v(wave);
        }
        for (uint32_t t = wave; t < tiles; t += kWaves) {
            const uint32_t bits = mask_of(t), next = t + kWaves, k = base + t * kOwnTile;
            wait_vmcnt<NP>();
            f32x16 s[1];
            w.scores(keys, s);
            wait_lgkm0();
            if (next < tiles) issue_k(next);
            const int64_t lim = sees - k;
            const uint32_t limit = lim < 0 ? 0u : lim > (int64_t)kOwnTile ? kOwnTile : (uint32_t)lim;
            const bool ragged = k + kOwnTile > common;
            if (ragged || bits != ~0u) w.mask(s, bits & ((1ull << limit) - 1ull));
            w.weights(scale, s);
            if (next < tiles) wait_vmcnt<NP>();
            else wait_vmcnt<0>();
            if (ragged && q_len > 1u)
                w.ragged_values(vals, s, valid ? limit : 0u, common > k ? common - k : 0u,
                                job.k1 - k < kOwnTile ? job.k1 - k : kOwnTile);
            typename Wave<T, DP>::Piece x[2][DP / 32];
            w.read_values(vals, 0, x[0]);
            w.values(vals, s, x);
            wait_lgkm0();
            if (next < tiles) issue_v(next);
        }
    }
    // join the waves
    cargs& e = fresh();
    constexpr uint32_t NF = DP / 8u;
    __syncthreads();
    float2* const ml = reinterpret_cast<float2*>(sh.kaddr);
    f32x4* const sums = reinterpret_cast<f32x4*>(sh.ring);
    const uint32_t tiles = (job.k1 - job.k0 + kOwnTile - 1u) / kOwnTile, busy = tiles < kWaves ? tiles : kWaves;
    const float total = w.total();
    if (lane < 32u) ml[wave * 32u + lane] = make_float2(w.m, total);
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
    for (uint32_t i = 0; i < busy; ++i) m = fmaxf(m, ml[i * 32u + n32].x);
    const float at = m == -INFINITY ? 0.0f : m;
    for (uint32_t i = 0; i < busy; ++i) l += ml[i * 32u + n32].y * __builtin_amdgcn_exp2f(ml[i * 32u + n32].x - at);
    if (wave < busy) {
        const float fade = __builtin_amdgcn_exp2f(w.m - at);
#pragma unroll
        for (uint32_t b = 0; b < DP / 32u; ++b)
#pragma unroll
            for (uint32_t g = 0; g < 4; ++g)
                sums[(wave * NF + 4u * b + g) * 64u + lane] =
                    f32x4{w.o[b][4u * g], w.o[b][4u * g + 1u], w.o[b][4u * g + 2u], w.o[b][4u * g + 3u]} * fade;
    }
    __syncthreads();
    f32x4* const out = part_at<DP>(e, job.block);
    for (uint32_t f = wave; f < NF; f += kWaves) {
        f32x4 x = (f32x4)(0.0f);
        for (uint32_t i = 0; i < busy; ++i) x += sums[(i * NF + f) * 64u + lane];
        if (!valid) continue;
        const uint32_t d = 8u * f + 4u * (lane / 32u);
        if (!e.direct) out[f * 64u + lane] = x;
        else if (d < e.dim) store_result<T>(e, job.head, r, d, l == 0.0f ? (f32x4)(0.0f) : x / l);
    }
    if (wave == 0 && valid && lane < 32u) {
        if (!e.direct) e.part_ml[job.block * 32u + lane] = make_float2(m, l);
        else if (e.lse) store_lse(e, job.head, r, m, l);
    }
}

template <typename T, uint32_t DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void k_attn(const AttnArgs) {
    cargs& a = kernel_args();
    __shared__ __attribute__((aligned(1024))) Shared<DP> sh;
    uint32_t id = blockIdx.x;
    OwnJob job;
    if (id < a.wg_all) {
        // Workgroups go to the 8 XCDs in turn: those that read the same part of
        // the prefix, one for each block of rows, meet in one XCD's L2, and so do
        // the heads of a part: where they lie side by side in a token's row, one
        // head alone would keep only two of the L2's 16 channels busy.
        const uint32_t rows = a.shared ? kWgRows : kRows, blocks = (a.rows_all + rows - 1u) / rows;
        const uint32_t x = id % 8u, y = id / 8u, each = (a.units_all + 7u) / 8u, unit = x * each + y / blocks;
        const uint32_t block = y % blocks;
        if (unit >= a.units_all) return;
        const uint32_t head = unit % a.kv, part = unit / a.kv;
        if (a.shared) return shared_part<T, DP>(a, sh, head, part, block);
        const uint32_t per = part_keys(a.prefix_len, a.parts_all, kOwnTile), left = a.rows_all - block * kRows;
        job.head = head;
        job.row = a.prefix_row;
        job.k0 = part_begin(a.prefix_len, part, per);
        job.k1 = part_begin(a.prefix_len, part + 1u, per);
        job.first = block * kRows;
        job.count = left < kRows ? left : kRows;
        job.len = 0;
        job.all = true;
        job.block = ((uint64_t)head * a.parts_all + part) * a.blocks_all + block;
    } else {
        id -= a.wg_all;
        job.head = id % a.kv;
        id /= a.kv;
        const uint32_t block = id % a.blocks_own;
        id /= a.blocks_own;
        const uint32_t part = id % a.parts_own, b = id / a.parts_own;
        job.row = a.rows ? (uint32_t)scalar_load(a.rows, b) : b;
        job.len = 0;
        if (job.row < a.table_rows) {
            const int64_t room = (int64_t)a.slots * a.row_pages, len = scalar_load(a.lens, job.row);
            job.len = len < 0 ? 0 : len > room ? room : len;
            if (job.len != len && threadIdx.x == 0) record_page_error(a.err);
        } else if (threadIdx.x == 0) {
            record_page_error(a.err);
        }
        const uint32_t per = part_keys((uint32_t)job.len, a.parts_own, kOwnTile), left = a.rows_own - block * kRows;
        job.k0 = part_begin((uint32_t)job.len, part, per);
        job.k1 = part_begin((uint32_t)job.len, part + 1u, per);
        job.first = b * a.rows_own + block * kRows;
        job.count = left < kRows ? left : kRows;
        job.all = false;
        job.block = a.own_first + (((uint64_t)b * a.kv + job.head) * a.blocks_own + block) * a.parts_own + part;
    }
    own_part<T, DP>(a, sh, job);
}

// The parts of 32 rows joined: blockIdx.x is the block of a head's rows, and
// each wave takes one piece of 8 elements of them.
template <typename T, uint32_t DP>
__global__ __launch_bounds__(kThreads) void k_attn_join(const AttnArgs) {
    cargs& a = kernel_args();
    constexpr uint32_t U = 16;                                            // parts in flight
    const uint32_t lane = lane_id(), n32 = lane % 32u, hh = lane / 32u;
    const uint32_t head = blockIdx.x / a.blocks_all, block = blockIdx.x - head * a.blocks_all;
    const uint32_t f = blockIdx.y * kWaves + threadIdx.x / 64u;
    const uint32_t d = 8u * f + 4u * hh;
    if (8u * f >= a.dim) return;
    uint32_t r = block * kRows + n32;
    const bool valid = r < a.rows_all;
    if (!valid) r = a.rows_all - 1u;
    const uint32_t b = r / a.rows_own, in = r - b * a.rows_own;
    const uint64_t own = a.own_first + (((uint64_t)b * a.kv + head) * a.blocks_own + in / kRows) * a.parts_own;
    const uint32_t parts = a.parts_all + a.parts_own;
    f32x4 acc = (f32x4)(0.0f);
    float m = -INFINITY, l = 0.0f;
    for (uint32_t i0 = 0; i0 < parts; i0 += U) {
        float2 ml[U];
        f32x4 x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            const uint32_t i = i0 + u;
            ml[u] = make_float2(-INFINITY, 0.0f);
            x[u] = (f32x4)(0.0f);
            if (i >= parts) continue;
            const bool all = i < a.parts_all;
            const uint64_t at = all ? ((uint64_t)head * a.parts_all + i) * a.blocks_all + block : own + (i - a.parts_all);
            const uint32_t slot = all ? n32 : in % kRows;
            ml[u] = a.part_ml[at * 32u + slot];
            x[u] = part_at<DP>(a, at)[f * 64u + hh * 32u + slot];
        }
        float next = m;
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) next = fmaxf(next, ml[u].x);
        const float at = next == -INFINITY ? 0.0f : next, fade = __builtin_amdgcn_exp2f(m - at);
        acc *= fade;
        l *= fade;
        m = next;
#pragma unroll
        for (uint32_t u = 0; u < U; ++u) {
            if (ml[u].y == 0.0f) continue;                                // a part that saw no key left no sums
            const float w = __builtin_amdgcn_exp2f(ml[u].x - at);
            l += w * ml[u].y;
            acc += x[u] * w;
        }
    }
    if (!valid) return;
    if (d < a.dim) store_result<T>(a, head, r, d, l == 0.0f ? (f32x4)(0.0f) : acc / l);
    if (f == 0 && hh == 0 && a.lse) store_lse(a, head, r, m, l);
}

// ---- host ---------------------------------------------------------------------------

// Shapes of the queries against a pool.
static bool shapes_fit(const View& q, const View& k) {
    return q.dim[0] == k.dim[0] && q.dim[0] % 8 == 0 && q.dim[0] <= 256 && q.dim[1] % k.dim[2] == 0 &&
           q.dim[1] <= 65535 && q.dim[2] <= 65535 && q.dim[3] <= 65535;
}

static uint32_t padded_dim(uint32_t dim) {
    return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256;
}

static uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// How the work is cut: fills the fields of `a` that follow from the shapes
// alone and returns the workspace's bytes, 0 if there are more rows than 31
// bits count or more workgroups than a launch holds.
static uint64_t plan(AttnArgs* a, uint64_t* groups_out) {
    constexpr uint64_t cus = 256;
    const uint64_t batch = (uint64_t)a->q.dim[3];
    const uint32_t dp = padded_dim((uint32_t)a->q.dim[0]);
    const uint64_t room = dp <= 128 ? 2 * cus : cus;                       // workgroups that run at once
    a->dim = (uint32_t)a->q.dim[0];
    a->q_len = (uint32_t)a->q.dim[2];
    a->kv = (uint32_t)a->k.dim[2];
    a->group = (uint32_t)a->q.dim[1] / a->kv;
    const uint64_t rows_own = (uint64_t)a->q_len * a->group, rows_all = rows_own * batch;
    if (rows_all > 0x7FFFFFFFull) return 0;
    a->rows_own = (uint32_t)rows_own;
    a->rows_all = (uint32_t)rows_all;
    a->blocks_own = (uint32_t)ceil_div(rows_own, kRows);
    a->blocks_all = (uint32_t)ceil_div(rows_all, kRows);
    // Four waves share the prefix's tiles where the product is large; otherwise
    // each has its own, which is read again for every 32 rows but needs no
    // meeting (8 key / value heads, own tiles first: 64 rows behind 16384 tokens
    // 24.4 and 25.3 us, 128 rows 31.1 and 28.2; 256 rows behind 4096 23.1 and
    // 26.2, 512 rows 37.4 and 32.1).
    a->shared = rows_all > 2 * kRows && a->kv * rows_all * a->prefix_len > 10000000;
    const uint64_t blocks = ceil_div(rows_all, a->shared ? kWgRows : kRows);
    // One workgroup on the prefix for each compute unit, so that the sequences'
    // own tokens are read beside it: two each are 17 % slower at 128 sequences
    // behind 32768 tokens, half as many 75 %.  Parts of 256 keys and above: each
    // is joined once more (64 rows behind 4096 tokens: parts of 128 keys 19.7 us,
    // 256 17.1, 512 18.8).
    a->parts_all = 0;
    if (a->prefix_len) {
        const uint64_t most = ceil_div(a->prefix_len, 256), want = cus / (a->kv * blocks);
        a->parts_all = (uint32_t)(want < 1 ? 1 : want < most ? want : most);
    }
    a->units_all = a->kv * a->parts_all;
    const uint64_t wg_all = ceil_div(a->units_all, 8) * 8 * blocks;
    const uint64_t jobs = batch * a->kv * a->blocks_own;
    // Without a prefix one part needs no second launch: 512 tokens of 64 elements
    // 9.8 us in one part and 11.3 in two, 1024 tokens 12.9 and 11.6 in four.
    const bool one = a->prefix_len == 0 && a->hint <= 512;
    const uint64_t most = one ? 1 : ceil_div(a->hint ? a->hint : 1, 256), want = room / jobs;
    a->parts_own = (uint32_t)(want < 1 ? 1 : want < most ? want : most);
    a->direct = a->parts_all == 0 && a->parts_own == 1;
    const uint64_t first = (uint64_t)a->units_all * a->blocks_all, own = jobs * a->parts_own;
    const uint64_t groups = wg_all + own;
    constexpr uint64_t most_groups = max_groups(kThreads);                 // of the products' launch, of the join's
    if (groups > most_groups || first > 0x7FFFFFFFull || (uint64_t)a->kv * a->blocks_all > most_groups) return 0;
    a->wg_all = (uint32_t)wg_all;
    a->own_first = (uint32_t)first;
    *groups_out = groups;
    const uint64_t parts = first + own;
    a->part_ml = reinterpret_cast<float2*>(parts * dp * 32 * 4);           // behind the sums
    return parts * (dp * 32 * 4 + 32 * 8) + 16;
}

template <typename T, uint32_t DP>
static tmap_status launch(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
    hipLaunchKernelGGL((k_attn<T, DP>), dim3(groups), dim3(kThreads), 0, stream, a);
    tmap_status st = check_launch("attn_shared_prefix");
    if (st || a.direct) return st;
    const dim3 grid(a.kv * a.blocks_all, (a.dim + 31u) / 32u);
    hipLaunchKernelGGL((k_attn_join<T, DP>), grid, dim3(kThreads), 0, stream, a);
    return check_launch("attn_shared_prefix");
}

template <typename T>
static tmap_status launch_dim(const AttnArgs& a, uint32_t groups, hipStream_t stream) {
    switch (padded_dim(a.dim)) {
    case 64: return launch<T, 64>(a, groups, stream);
    case 96: return launch<T, 96>(a, groups, stream);
    case 128: return launch<T, 128>(a, groups, stream);
    case 192: return launch<T, 192>(a, groups, stream);
    default: return launch<T, 256>(a, groups, stream);
    }
}

}  // namespace att

using namespace att;

extern "C" uint64_t attn_workspace(const tmap_t* q, const tmap_t* k_pool, uint32_t prefix_len,
                                   uint32_t suffix_hint) {
    AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    int32_t tq, tk;
    if (view_of(q, 4, &a.q, &tq) || view_of(k_pool, 4, &a.k, &tk) || !shapes_fit(a.q, a.k)) return 0;
    a.prefix_len = prefix_len;
    a.hint = suffix_hint;
    uint64_t groups;
    return plan(&a, &groups);
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
        (uint64_t)a.k.dim[1] != pt->slots || (uint64_t)a.k.dim[3] != pt->pages || !std::isfinite(scale * kLog2e))
        return TMAP_ERR_UNSUPPORTED;
    if (prefix_len && (prefix_row >= pt->rows || prefix_len > (uint64_t)pt->slots * pt->row_pages))
        return TMAP_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(d_ws) % 16 != 0) return TMAP_ERR_ALIGN;
    a.prefix_len = prefix_len;
    a.hint = suffix_hint;
    uint64_t groups = 0;
    const uint64_t need = plan(&a, &groups);
    if (need == 0 || ws_bytes < need) return TMAP_ERR_UNSUPPORTED;
    a.part_o = static_cast<f32x4*>(d_ws);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(d_ws) + reinterpret_cast<uintptr_t>(a.part_ml));
    a.table = pt->d_table;
    a.lens = pt->d_lens;
    a.rows = d_rows;
    a.pitch = pt->pitch;
    a.table_rows = pt->rows;
    a.row_pages = pt->row_pages;
    a.pages = pt->pages;
    a.slots = pt->slots;
    a.prefix_row = prefix_row;
    // Scores are kept in powers of two.  A negative scale turns the queries
    // around and a scale of 0 makes them 0, so that the factor is above 0 and
    // masked scores stay at -inf.
    a.zero = scale == 0;
    a.scale = a.zero ? 1.0f : std::fabs(scale) * kLog2e;
    a.flip = scale < 0 ? 0x80008000u : 0u;
    a.lse = d_lse;
    st = device_error_word(&a.err);
    if (st) return st;
    if (tq == TMAP_F16) return launch_dim<_Float16>(a, (uint32_t)groups, as_stream(stream));
    return launch_dim<__bf16>(a, (uint32_t)groups, as_stream(stream));
}
