// attn_wave.hpp -- what the attention kernels are made of: a wave's 32 queries
// on the matrix cores, tiles of keys and values in LDS and the copies that fill
// them.
//
// Scores are computed transposed, keys x queries (A = keys from LDS, B = queries
// in registers), so that a lane owns one query and the maximum and the sum over
// keys stay inside it, up to one exchange with the lane 32 further.  The weights,
// rounded to the element type, then already lie as the second product's B operand
// (values transposed x weights) if that product takes its keys in the order 0-3,
// 8-11 | 4-7, 12-15, which the transposing LDS read of the values delivers for
// free.
#pragma once

#include <hip/hip_runtime.h>

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
// Powers of two by which weights are taken larger for f16, whose smallest number is
// 2^-24: with it a weight vanishes below 2^-32 of the largest one, not below 2^-25
// (131072 tokens 17.5 below the largest score are 0.3 % of a result).  They may pass the
// largest of before by 2^7 then, not by 2^kLazy: 2^14 times the rest of a scale, below
// 2, leaves a factor of two for the roundings of scores, in powers of two, up to 2^24.
constexpr float kHead = 7.0f;
constexpr float kHeadLazy = 7.0f;

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

// A wave's 32 queries and what it has summed for them.  Lane l: query l % 32,
// half l / 32 of each group of 8 keys (scores) or 8 elements (result).
// AGAIN: offsets within a tile are worked out for each tile.  Kept from tile to tile,
// beside codes on their way, they do not fit into the registers, and one that comes
// back from memory waits for the codes too (2048 queries of 32768 e4m3 tokens: 1247 us,
// this 1165).
// HEAD: f16 weights are taken 2^kHead times as large.
template <typename T, uint32_t DP, bool AGAIN = false, bool HEAD = false>
struct Wave {
    typedef typename Vec<T>::v8 v8;
    typedef typename Vec<T>::v4 v4;
    static constexpr bool headed = HEAD && std::is_same<T, _Float16>::value;
    static constexpr float head = headed ? kHead : 0.0f, most = headed ? kHead + kHeadLazy : kLazy;
    static constexpr uint32_t NK = DP / 16, NO = DP / 32;
    v8 q[NK];
    f32x16 o[NO];
    float m, l;                      // largest score seen, in powers of two, less head (or less: lazily), sum of weights

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
    template <class Args>
    __device__ __forceinline__ void load(const Args& a, uint32_t head, uint32_t r, bool valid) {
        const uint32_t b = r / a.rows_own, in = r - b * a.rows_own, j = in / a.group, g = in - j * a.group;
        load_row(a, gptr(a.q.base) + (int64_t)b * a.q.stride[3] + (int64_t)j * a.q.stride[2] +
                        (int64_t)(head * a.group + g) * a.q.stride[1], valid);
    }

    // The lane's query at p.
    template <class Args>
    __device__ __forceinline__ void load_row(const Args& a, const gbyte* p, bool valid) {
        const uint32_t lane = lane_id();
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
        const uint32_t lane = lane_id(), row = lane % 32u;
        const uint8_t* at = keys + row * (DP * 2u);
        uint32_t chunk = (lane / 32u ^ Geo<DP>::key_k(row)) * 16u;
        if (AGAIN) asm volatile("" : "+v"(chunk));
        v8 x[AHEAD + 1][NB];
        auto read = [&](uint32_t k) {
#pragma unroll
            for (uint32_t n = 0; n < NB; ++n)
                x[k % (AHEAD + 1)][n] = *reinterpret_cast<const v8*>(at + n * 32u * (DP * 2u) + (32u * k ^ chunk));
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
    // 2^kLazy; weights then stay below 2^most, which both types hold.
    // Returns what weights are taken relative to.  Each query goes by its own
    // scores, so its result does not depend on the others of the wave.  A top
    // that is NaN (no score is a number) makes the sums NaN, as it has to.
    __device__ __forceinline__ float rescale(float top) {
        const bool pass = !(top <= m + most);
        if (__any(pass)) {
            const float next = top - head, fade = pass ? __builtin_amdgcn_exp2f(m - next) : 1.0f;
            m = pass ? next : m;
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
        const uint32_t c0 = 2u * ((lane / 16u) & 1u) + (i % 4u) / 2u;
        const uint8_t* at = vals + (step * 16u + row) * (DP * 2u) + 8u * (i & 1u);
        uint32_t chunk = (c0 ^ Geo<DP>::key_v(row)) * 16u;
        if (AGAIN) asm volatile("" : "+v"(chunk));
#pragma unroll
        for (uint32_t b = 0; b < NO; ++b) {
            const uint8_t* v = at + (64u * b ^ chunk);
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
    // Returns the largest of the next scores.  KEYS, VALUES: the next scores are
    // multiplied by scales of their keys, this tile's weights (but not their sum)
    // by scales of theirs.  FREE: the compiler may move instructions from one product
    // to another.
    template <bool KEYS = false, bool VALUES = false, bool FREE = false>
    __device__ __forceinline__ float advance(float scale, const uint8_t* keys, const uint8_t* vals, float top,
                                             f32x16 (&s)[2], f32x16 (&next)[2], const float* key_scales = nullptr,
                                             const float* value_scales = nullptr) {
        // Products of scores, of values, and how far ahead of them LDS is read.  Beside
        // scales and codes on their way, what is read five ahead does not fit into the
        // registers (2048 queries of 32768 e4m3 tokens: 1695 us, three ahead 1505, two 1247).
        constexpr uint32_t NS = 2 * NK, NP = 4 * NO, AHEAD = KEYS ? 2 : 5;
        const uint32_t lane = lane_id(), row = lane % 32u;
        const uint32_t i16 = lane % 16u, vrow = 4u * (lane / 32u) + i16 / 4u;
        const uint32_t c0 = 2u * ((lane / 16u) & 1u) + (i16 % 4u) / 2u;
        const uint8_t* kat = keys + row * (DP * 2u);
        const uint8_t* vat = vals + vrow * (DP * 2u) + 8u * (i16 & 1u);
        uint32_t kchunk = (lane / 32u ^ Geo<DP>::key_k(row)) * 16u, vchunk = (c0 ^ Geo<DP>::key_v(vrow)) * 16u;
        if (AGAIN) asm volatile("" : "+v"(kchunk), "+v"(vchunk));
        Piece x[AHEAD + 1];
        auto read = [&](uint32_t i) {                                     // what product i takes from LDS
            Piece& y = x[i % (AHEAD + 1u)];
            if (i < NS) {
                const uint32_t k = i / 2u, n = i % 2u;
                y.v = *reinterpret_cast<const v8*>(kat + n * 32u * (DP * 2u) + (32u * k ^ kchunk));
            } else if (i < NS + NP) {
                const uint32_t t = (i - NS) / NO, b = (i - NS) % NO;
                const uint8_t* v = vat + t * 16u * (DP * 2u) + (64u * b ^ vchunk);
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
        f32x4 ks[2], vs[2];                                               // of 4 keys each, read 4 keys ahead
        const float* const ksat = key_scales + 4u * (lane / 32u);
        const float* const vsat = value_scales + 4u * (lane / 32u);
        if (VALUES) vs[0] = *reinterpret_cast<const f32x4*>(vsat);
        static_for<(int)(NS + NP)>([&](auto slot) {
            constexpr uint32_t i = decltype(slot)::value;
            read(i + AHEAD);
            if constexpr (KEYS && i == NS) ks[0] = *reinterpret_cast<const f32x4*>(ksat);
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
                if constexpr (VALUES && e % 4u == 0 && e + 4u < 32u)
                    vs[(e / 4u + 1u) & 1u] = *reinterpret_cast<const f32x4*>(vsat + 2u * (e + 4u));
                w[e / 8u][e % 8u] = (T)(VALUES ? p * vs[e / 4u & 1u][e % 4u] : p);
            });
            // the next scores' largest, from the third product of values on
            constexpr uint32_t per = (32u + NP - 3u) / (NP - 2u), j0 = i < NS + 2u ? 32u : (i - NS - 2u) * per;
            static_for<(int)(j0 < 32u ? (32u - j0 < per ? 32u - j0 : per) : 0u)>([&](auto which) {
                constexpr uint32_t j = j0 + decltype(which)::value;
                if constexpr (KEYS) {
                    if constexpr (j % 4u == 0 && j + 4u < 32u)
                        ks[(j / 4u + 1u) & 1u] = *reinterpret_cast<const f32x4*>(ksat + 2u * (j + 4u));
                    next[j / 16u][j % 16u] *= ks[j / 4u & 1u][j % 4u];
                }
                if constexpr (j == 0) best = next[0][0];
                else best = fmaxf(best, next[j / 16u][j % 16u]);
            });
            if constexpr (!FREE) __builtin_amdgcn_sched_barrier(0);
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

    // Whether share `part` of `parts` of a tile of `rows` values holds infinities
    // or NaN (CLEAR: and those become 0); the same in every lane of the wave.
    template <bool CLEAR>
    __device__ __forceinline__ static bool odd_share(uint8_t* vals, uint32_t part, uint32_t parts, uint32_t rows) {
        bool odd = false;
        for (uint32_t i = part * 64u + lane_id(); i < rows * Geo<DP>::cpr; i += parts * 64u) {
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

    // The infinities and NaN among a tile's values, added to the rows that see
    // their keys (a bit of `sees` each).
    template <uint32_t NB>
    __device__ __forceinline__ void add_odd(const uint8_t* vals, const f32x16 (&p)[NB], uint64_t sees) {
        const uint32_t hh = lane_id() / 32u;
        for (uint32_t key = 0; key < 32u * NB; ++key) {
            const uint32_t at = 4u * (key % 32u / 8u) + key % 4u;
            float x = 0.0f;
#pragma unroll
            for (uint32_t n = 0; n < NB; ++n)
#pragma unroll
                for (uint32_t i = 0; i < 16; ++i)
                    if (n == key / 32u && i == at && (key >> 2 & 1u) == hh) x = p[n][i];
            x = (float)(T)add_halves(x);
            const uint8_t* row = vals + key * (DP * 2u) + 8u * hh;
#pragma unroll
            for (uint32_t f = 0; f < DP / 8u; ++f) {
                const uint64_t bits = *reinterpret_cast<const uint64_t*>(row + (f ^ Geo<DP>::key_v(key)) * 16u);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) {
                    const uint16_t h = (uint16_t)(bits >> (16u * e));
                    if (not_finite(h) && (sees >> key & 1u))
                        o[f / 4u][4u * (f % 4u) + e] += x * (float)__builtin_bit_cast(T, h);
                }
            }
        }
    }

    // Sum of the weights over both halves.
    __device__ __forceinline__ float total() const { return add_halves(l); }
};

// Copy n of N of a wave's share of a tile: groups first, first + STEP, ... of
// 64 chunks each.  Chunk i = 64 * group + lane is row i / cpr; the row's
// address says where it lies.  FULL: the row has DP elements.
template <uint32_t DP, uint32_t STEP, bool VALUES, bool FULL = false>
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
        if constexpr (FULL) return at;
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

}  // namespace att
