// kernel_rope.hip -- rotary positions: the plan's encoder, the rotation of a
// tensor of heads, and the step that writes a token's keys and values to
// their page.
//
// Pair j of a head turns by position * theta_j.  The plan holds theta_j / 2 pi
// (turns per position) in 64 bits; a kernel takes the product with the
// position as an exact two-term sum (product and its rounding error, one fma),
// drops the whole turns and only then goes to fp32, so that the fraction of a
// turn is right to fp32 precision at any int32 position.
//
// Bound: HBM, or the launch for a few tokens.  A head's element is read once
// and written once; the cosine and sine of a (token, pair) are computed once
// per workgroup, into LDS, and used for every head of the token.  8192 tokens of
// 32 x 128 bf16 take 22.2 us (6.0 TB/s), the step that writes 8191 tokens' keys and
// values to their pages 38.3 us (5.2 TB/s); 64 tokens' step 8.3 us, of which the
// kernel is 6.8.  Short of 32 MiB the layouts differ: 4096 tokens (67 MB, 12.9 us at
// 5.2 TB/s) take 13.7 us in pairs side by side, 16.5 in halves of the whole head,
// 17.9 to 18.8 with part of the head turned (lanes with two chunks of a pair beside
// lanes with one of the rest), 21.3 to 21.8 element by element.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "cache_util.hpp"

namespace att {

constexpr uint32_t kMaxPairs = 128;
constexpr uint32_t kRopeThreads = 256;
constexpr uint32_t kTokMax = 2;         // tokens of a workgroup

struct RopePlan {
    double turns[kMaxPairs];   // turns per position of each pair
    float magnitude;
    uint32_t rot;              // rotated elements of a head
    int32_t layout;
    uint32_t pad[9];
};
static_assert(sizeof(RopePlan) == sizeof(rope_t), "the plan fills the public type");

// One tensor of the call: heads that are rotated (or copied) from src to dst.
struct RopeSeg {
    uint64_t src, dst;
    int64_t src_head, src_tok;      // byte strides
    int64_t dst_head, dst_tok;      // dst_tok: of a slot for a pool
    int64_t dst_page;               // 0: dst is a tensor, else of a page
    uint32_t heads;
    uint32_t rotate;
};

// The plan's frequencies as a kernel takes them.  A launch costs the host about
// 0.7 us more for each KiB of arguments, so a small call passes only as many as
// it needs.
template <uint32_t P>
struct RopeTurns {
    double turns[P];
};

struct RopeArgs {
    RopeSeg seg[3];
    const int32_t* pos;
    const int32_t* rows;            // pools: row and token index of each token
    const int32_t* at;
    const int32_t* table;
    uint64_t pitch;
    uint32_t* err;
    float magnitude, sine;          // of the cosine and the sine (whose sign turns for the inverse)
    uint32_t rot;
    uint32_t nseg, tokens, dim;
    uint32_t table_rows, row_pages, pages, slots;
    uint32_t units, tok_block, head_lanes;
    uint32_t in_place;
};

// How a thread's unit of a head is formed.
//   PAIRED    one 16-byte chunk, pairs side by side in it
//   SPLIT     two 16-byte chunks, rot / 2 elements apart (rot / 2 a whole
//             number of chunks), or one chunk past rot
//   ELEMENTS  one pair, or one element past rot: ROPE_HALF with halves that
//             are not whole chunks
enum { PAIRED = 0, SPLIT = 1, ELEMENTS = 2 };

template <typename T>
struct Chunk {
    static constexpr uint32_t N = 16 / sizeof(T);
    T e[N];
};

template <typename T>
__device__ __forceinline__ void load_chunk(Chunk<T>& c, const gbyte* p, uint32_t n) {
    if (n == Chunk<T>::N) {
        const u32x4 v = *(const ATT_GLOBAL u32x4*)p;
        __builtin_memcpy(&c, &v, 16);
    } else {
#pragma unroll
        for (uint32_t i = 0; i < Chunk<T>::N; ++i)
            if (i < n) c.e[i] = ((const ATT_GLOBAL T*)p)[i];
    }
}

template <bool STREAM, typename T>
__device__ __forceinline__ void store_chunk(const Chunk<T>& c, gbyte* p, uint32_t n) {
    if (n == Chunk<T>::N) {
        u32x4 v;
        __builtin_memcpy(&v, &c, 16);
        if (STREAM) __builtin_nontemporal_store(v, (ATT_GLOBAL u32x4*)p);
        else *(ATT_GLOBAL u32x4*)p = v;
    } else {
#pragma unroll
        for (uint32_t i = 0; i < Chunk<T>::N; ++i)
            if (i < n) ((ATT_GLOBAL T*)p)[i] = c.e[i];
    }
}

// STREAM: the call writes more than the L2s hold, so its output is not kept
// there.
template <typename T, int MODE, bool STREAM, uint32_t P>
__global__ __launch_bounds__(kRopeThreads) void k_rope(const RopeTurns<P> plan, const RopeArgs a) {
    constexpr uint32_t N = Chunk<T>::N;
    __shared__ float2 turn[kTokMax][P];           // magnitude * (cos, sin)
    __shared__ int2 where[kTokMax];               // page (-1: none) and slot
    const uint32_t tid = threadIdx.x;
    const uint32_t t0 = blockIdx.x * a.tok_block;
    const uint32_t pairs = a.rot / 2;
    for (uint32_t i = tid; i < a.tok_block * pairs; i += kRopeThreads) {
        const uint32_t k = i / pairs, j = i - k * pairs;
        if (t0 + k < a.tokens) {
            const double p = (double)a.pos[t0 + k], f = plan.turns[j];
            const double whole = p * f;
            const double part = (whole - rint(whole)) + fma(p, f, -whole);
            float s, c;
            sincospif(2.0f * (float)part, &s, &c);
            turn[k][j] = make_float2(a.magnitude * c, a.sine * s);
        }
    }
    if (a.table && tid < a.tok_block && t0 + tid < a.tokens) {
        const int32_t row = a.rows[t0 + tid], at = a.at[t0 + tid];
        int2 w = make_int2(-1, 0);
        if (row >= 0) {
            const uint32_t col = (uint32_t)at / a.slots;
            if ((uint32_t)row < a.table_rows && at >= 0 && col < a.row_pages) {
                const int32_t page = a.table[(uint64_t)(uint32_t)row * a.pitch + col];
                if ((uint32_t)page < a.pages) w = make_int2(page, (int32_t)((uint32_t)at - col * a.slots));
            }
            if (w.x < 0) record_page_error(a.err);
        }
        where[tid] = w;
    }
    __syncthreads();

    const uint32_t u = tid % a.units, hl = (tid / a.units) % a.head_lanes, k = tid / (a.units * a.head_lanes);
    if (k >= a.tok_block || t0 + k >= a.tokens) return;
    const uint32_t t = t0 + k;

    // the unit's elements: [e0, e0 + n0), and the partners [e1, e1 + n0)
    const uint32_t per = MODE == ELEMENTS ? 1u : N;
    uint32_t e0, e1 = 0, pair0;
    bool turned, two;
    if (MODE == PAIRED) {
        e0 = u * N;
        pair0 = e0 / 2;
        turned = e0 < a.rot;
        two = false;
    } else {
        const uint32_t half = pairs / per;                // units that hold a pair
        two = u < half;
        e0 = two ? u * per : a.rot + (u - half) * per;
        e1 = e0 + pairs;
        pair0 = e0;
        turned = two;
    }
    const uint32_t n0 = a.dim - e0 < per ? a.dim - e0 : per;
    float cs[N], sn[N];
    if (turned) {
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) {
            if (i >= per) break;
            const uint32_t j = MODE == PAIRED ? pair0 + i / 2 : pair0 + i;
            const float2 v = j < pairs ? turn[k][j] : make_float2(1.0f, 0.0f);
            cs[i] = v.x;
            sn[i] = v.y;
        }
    }

    constexpr uint32_t U = 4;                             // heads in flight per thread
    for (uint32_t s = 0; s < a.nseg; ++s) {
        const RopeSeg& g = a.seg[s];
        int64_t off = (int64_t)t * g.dst_tok;
        if (g.dst_page) {
            const int2 w = where[k];
            if (w.x < 0) continue;
            off = (int64_t)w.x * g.dst_page + (int64_t)w.y * g.dst_tok;
        }
        const gbyte* src = gptr(g.src) + (int64_t)t * g.src_tok;
        gbyte* dst = gptr(g.dst) + off;
        const bool rot = turned && g.rotate;
        if (!rot && a.in_place) continue;                 // the elements stay where they are
        for (uint32_t h0 = hl; h0 < g.heads; h0 += U * a.head_lanes) {
            Chunk<T> x[U], y[U];
#pragma unroll
            for (uint32_t i = 0; i < U; ++i) {
                const uint32_t h = h0 + i * a.head_lanes;
                if (h < g.heads) {
                    const gbyte* p = src + (int64_t)h * g.src_head;
                    if (MODE == ELEMENTS) {
                        x[i].e[0] = ((const ATT_GLOBAL T*)p)[e0];
                        if (two) y[i].e[0] = ((const ATT_GLOBAL T*)p)[e1];
                    } else {
                        load_chunk(x[i], p + e0 * sizeof(T), n0);
                        if (two) load_chunk(y[i], p + e1 * sizeof(T), N);
                    }
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < U; ++i) {
                const uint32_t h = h0 + i * a.head_lanes;
                if (h >= g.heads) break;
                if (rot) {
                    if (MODE == PAIRED) {
#pragma unroll
                        for (uint32_t q = 0; q < N; q += 2) {
                            if (pair0 + q / 2 < pairs) {
                                const float f = (float)x[i].e[q], l = (float)x[i].e[q + 1];
                                x[i].e[q] = (T)(f * cs[q] - l * sn[q]);
                                x[i].e[q + 1] = (T)(f * sn[q] + l * cs[q]);
                            }
                        }
                    } else {
#pragma unroll
                        for (uint32_t q = 0; q < N; ++q) {
                            if (q >= per) break;
                            const float f = (float)x[i].e[q], l = (float)y[i].e[q];
                            x[i].e[q] = (T)(f * cs[q] - l * sn[q]);
                            y[i].e[q] = (T)(f * sn[q] + l * cs[q]);
                        }
                    }
                }
                gbyte* p = dst + (int64_t)h * g.dst_head;
                if (MODE == ELEMENTS) {
                    ((ATT_GLOBAL T*)p)[e0] = x[i].e[0];
                    if (two) ((ATT_GLOBAL T*)p)[e1] = y[i].e[0];
                } else {
                    store_chunk<STREAM>(x[i], p + e0 * sizeof(T), n0);
                    if (two) store_chunk<STREAM>(y[i], p + e1 * sizeof(T), N);
                }
            }
        }
    }
}

// The arguments of the tokens behind the first n.
static void skip_tokens(RopeArgs& a, uint32_t n) {
    for (uint32_t i = 0; i < a.nseg; ++i) {
        a.seg[i].src += (uint64_t)n * (uint64_t)a.seg[i].src_tok;
        if (!a.seg[i].dst_page) a.seg[i].dst += (uint64_t)n * (uint64_t)a.seg[i].dst_tok;
    }
    if (a.pos) a.pos += n;
    if (a.rows) a.rows += n, a.at += n;
}

template <typename T, int MODE, bool STREAM, uint32_t P>
static void launch_pairs(const RopePlan& plan, const RopeArgs& a, hipStream_t stream) {
    RopeTurns<P> turns;
    std::memcpy(&turns, plan.turns, sizeof(turns));
    constexpr uint32_t most = max_groups(kRopeThreads);
    RopeArgs part = a;
    for (uint32_t left = a.tokens; left; left -= part.tokens) {
        const uint32_t groups = (left - 1) / a.tok_block + 1;
        part.tokens = groups <= most ? left : most * a.tok_block;
        const dim3 grid((part.tokens - 1) / a.tok_block + 1);
        hipLaunchKernelGGL((k_rope<T, MODE, STREAM, P>), grid, dim3(kRopeThreads), 0, stream, turns, part);
        skip_tokens(part, part.tokens);
    }
}

template <typename T, int MODE>
static void launch_size(const RopePlan& plan, const RopeArgs& a, bool stream_out, hipStream_t stream) {
    if (stream_out) launch_pairs<T, MODE, true, kMaxPairs>(plan, a, stream);
    else if (a.rot <= 64) launch_pairs<T, MODE, false, 32>(plan, a, stream);
    else if (a.rot <= 128) launch_pairs<T, MODE, false, 64>(plan, a, stream);
    else launch_pairs<T, MODE, false, kMaxPairs>(plan, a, stream);
}

template <typename T>
static void launch_mode(const RopePlan& plan, RopeArgs& a, hipStream_t stream) {
    constexpr uint32_t N = 16 / sizeof(T);
    const uint32_t rot = a.rot, rest = a.dim - rot;
    int mode;
    if (plan.layout == ROPE_INTERLEAVED) {
        mode = PAIRED;
        a.units = (a.dim + N - 1) / N;
    } else if (rot / 2 % N == 0) {
        mode = SPLIT;
        a.units = rot / 2 / N + (rest + N - 1) / N;
    } else {
        mode = ELEMENTS;
        a.units = rot / 2 + rest;
    }
    // Tokens of a workgroup: two, which share its start, once each thread has
    // work for them (8192 tokens of 32 x 128 bf16: 25.7 us with one, 24.2 with
    // two, 25.9 with eight), but one each while there are too few to fill the GPU.
    const uint32_t most = a.units > rot / 2 ? a.units : rot / 2;
    a.tok_block = most > kRopeThreads / 2 || a.tokens < 1024u ? 1u : kTokMax;
    a.head_lanes = kRopeThreads / (a.units * a.tok_block);
    // Beyond the L2s (8 x 4 MiB) the output is streamed: 8192 tokens as above
    // 31 -> 26 us, the write of 8191 tokens to their pages 48 -> 43 us.
    uint64_t heads = 0;
    for (uint32_t i = 0; i < a.nseg; ++i) heads += a.seg[i].heads;
    const bool stream_out = heads * a.tokens * a.dim * sizeof(T) > (32ull << 20);
    if (mode == PAIRED) launch_size<T, PAIRED>(plan, a, stream_out, stream);
    else if (mode == SPLIT) launch_size<T, SPLIT>(plan, a, stream_out, stream);
    else launch_size<T, ELEMENTS>(plan, a, stream_out, stream);
}

static tmap_status launch_rope(const RopePlan& plan, RopeArgs& a, bool inverse, int32_t dtype, void* stream,
                               const char* name) {
    a.rot = plan.rot;
    a.magnitude = plan.magnitude;
    a.sine = inverse ? -plan.magnitude : plan.magnitude;
    switch (dtype) {
    case TMAP_F16: launch_mode<_Float16>(plan, a, as_stream(stream)); break;
    case TMAP_BF16: launch_mode<__bf16>(plan, a, as_stream(stream)); break;
    default: launch_mode<float>(plan, a, as_stream(stream)); break;
    }
    return check_launch(name);
}

static RopePlan load_plan(const rope_t* r) {
    RopePlan p;
    std::memcpy(&p, r, sizeof(p));
    return p;
}

static bool rope_type(int32_t dtype) { return dtype == TMAP_F16 || dtype == TMAP_BF16 || dtype == TMAP_F32; }

// Shape limits of a tensor of heads {dim, heads, tokens} under a plan.
static bool heads_fit(const View& v, uint32_t rot) {
    return v.dim[0] >= rot && v.dim[0] <= 256 && v.dim[1] <= 65535 && v.dim[2] <= 0x7FFFFFFF;
}

static RopeSeg tensor_seg(const View& x, const View& y) {
    return {x.base, y.base, x.stride[1], x.stride[2], y.stride[1], y.stride[2], 0, (uint32_t)x.dim[1], 1u};
}

static RopeSeg pool_seg(const View& x, const View& pool, bool rotate) {
    return {x.base, pool.base, x.stride[1], x.stride[2], pool.stride[2], pool.stride[1], pool.stride[3],
            (uint32_t)x.dim[1], rotate ? 1u : 0u};
}

}  // namespace att

using namespace att;

extern "C" tmap_status rope_encode(rope_t* out, uint32_t rot_dim, int32_t layout, double base, int32_t scaling,
                                   double factor, uint32_t original_len, double slow, double fast,
                                   double magnitude) {
    if (!out) return TMAP_ERR_NULL;
    std::memset(out, 0, sizeof(*out));
    if (rot_dim < 2 || rot_dim > 2 * kMaxPairs || rot_dim % 2 != 0) return TMAP_ERR_UNSUPPORTED;
    if (layout != ROPE_HALF && layout != ROPE_INTERLEAVED) return TMAP_ERR_UNSUPPORTED;
    if (scaling < ROPE_SCALE_NONE || scaling > ROPE_SCALE_RAMP) return TMAP_ERR_UNSUPPORTED;
    if (!(base > 0) || !std::isfinite(base) || !std::isfinite((float)magnitude)) return TMAP_ERR_UNSUPPORTED;
    if (scaling != ROPE_SCALE_NONE && (!(factor > 0) || !std::isfinite(factor))) return TMAP_ERR_UNSUPPORTED;
    if (scaling == ROPE_SCALE_RAMP &&
        (original_len == 0 || !(fast > slow) || !std::isfinite(fast) || !std::isfinite(slow)))
        return TMAP_ERR_UNSUPPORTED;
    RopePlan p;
    std::memset(&p, 0, sizeof(p));
    p.rot = rot_dim;
    p.layout = layout;
    p.magnitude = (float)magnitude;
    if (scaling == ROPE_SCALE_BASE && rot_dim > 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return TMAP_ERR_UNSUPPORTED;
    const double two_pi = 6.283185307179586476925286766559;
    for (uint32_t j = 0; j < rot_dim / 2; ++j) {
        double theta = std::pow(base, -2.0 * j / rot_dim);
        if (scaling == ROPE_SCALE_LINEAR) theta /= factor;
        if (scaling == ROPE_SCALE_RAMP) {
            double w = (original_len * theta / two_pi - slow) / (fast - slow);
            w = w < 0 ? 0 : w > 1 ? 1 : w;
            theta *= w + (1 - w) / factor;
        }
        p.turns[j] = theta / two_pi;
        if (!std::isfinite(p.turns[j] * 2147483648.0)) return TMAP_ERR_UNSUPPORTED;   // the farthest position
    }
    std::memcpy(out, &p, sizeof(p));
    return TMAP_OK;
}

extern "C" tmap_status rope_apply(const rope_t* r, const tmap_t* x, const tmap_t* y, const int32_t* d_pos,
                                  int32_t inverse, void* stream) {
    if (!r || !x || !y || !d_pos) return TMAP_ERR_NULL;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    View vx, vy;
    int32_t tx, ty;
    tmap_status st = view_of(x, 3, &vx, &tx);
    if (st == TMAP_OK) st = view_of(y, 3, &vy, &ty);
    if (st) return st;
    if (!rope_type(tx)) return TMAP_ERR_DTYPE;
    const RopePlan plan = load_plan(r);
    if (ty != tx || !same_dims(vx, vy) || plan.rot < 2 || !heads_fit(vx, plan.rot)) return TMAP_ERR_UNSUPPORTED;
    a.in_place = vx.base == vy.base;
    if (a.in_place && (vx.stride[1] != vy.stride[1] || vx.stride[2] != vy.stride[2])) return TMAP_ERR_UNSUPPORTED;
    a.seg[0] = tensor_seg(vx, vy);
    a.nseg = 1;
    a.pos = d_pos;
    a.tokens = (uint32_t)vx.dim[2];
    a.dim = (uint32_t)vx.dim[0];
    return launch_rope(plan, a, inverse != 0, tx, stream, "rope_apply");
}

extern "C" tmap_status rope_append(const rope_t* r, const tmap_t* q, const tmap_t* q_out, const tmap_t* k,
                                   const tmap_t* v, const tmap_t* k_pool, const tmap_t* v_pool,
                                   const page_table_t* pt, const int32_t* d_rows, const int32_t* d_at,
                                   const int32_t* d_pos, void* stream) {
    if (!k || !v || !k_pool || !v_pool || !pt || !d_rows || !d_at) return TMAP_ERR_NULL;
    if ((r && !d_pos) || (q != nullptr) != (q_out != nullptr)) return TMAP_ERR_NULL;
    RopeArgs a;
    std::memset(&a, 0, sizeof(a));
    View vk, vv, pk, pv;
    int32_t tk, tv, tpk, tpv;
    tmap_status st = view_of(k, 3, &vk, &tk);
    if (st == TMAP_OK) st = view_of(v, 3, &vv, &tv);
    if (st == TMAP_OK) st = view_of(k_pool, 4, &pk, &tpk);
    if (st == TMAP_OK) st = view_of(v_pool, 4, &pv, &tpv);
    if (st == TMAP_OK) st = check_table(pt);
    if (st) return st;
    if (!rope_type(tk)) return TMAP_ERR_DTYPE;
    RopePlan plan;
    std::memset(&plan, 0, sizeof(plan));
    if (r) plan = load_plan(r);
    if (r && plan.rot < 2) return TMAP_ERR_UNSUPPORTED;
    if (tv != tk || tpk != tk || tpv != tk || !same_dims(vk, vv) || !same_dims(pk, pv) ||
        !heads_fit(vk, plan.rot) || pk.dim[0] != vk.dim[0] || pk.dim[2] != vk.dim[1] ||
        pk.dim[1] != pt->slots || pk.dim[3] != pt->pages)
        return TMAP_ERR_UNSUPPORTED;
    if (q) {
        View vq, vo;
        int32_t tq, to;
        st = view_of(q, 3, &vq, &tq);
        if (st == TMAP_OK) st = view_of(q_out, 3, &vo, &to);
        if (st) return st;
        if (tq != tk || to != tk || !same_dims(vq, vo) || !heads_fit(vq, plan.rot) || vq.dim[0] != vk.dim[0] ||
            vq.dim[2] != vk.dim[2])
            return TMAP_ERR_UNSUPPORTED;
        if (vq.base == vo.base && (vq.stride[1] != vo.stride[1] || vq.stride[2] != vo.stride[2]))
            return TMAP_ERR_UNSUPPORTED;
        a.seg[a.nseg++] = tensor_seg(vq, vo);
    }
    a.seg[a.nseg++] = pool_seg(vk, pk, r != nullptr);
    a.seg[a.nseg++] = pool_seg(vv, pv, false);
    a.pos = d_pos;
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
    st = device_error_word(&a.err);
    if (st) return st;
    return launch_rope(plan, a, false, tk, stream, "rope_append");
}
