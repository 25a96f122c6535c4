// kernel_attn_cache.hip -- attention over the cache: the parts joined, and the
// calls.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "attn_cache.hpp"

namespace att {

// The parts of 32 rows joined: blockIdx.x is the block of a sequence's head.  Each wave
// takes one piece of 8 elements of them, or (SPLIT) a workgroup does, whose waves
// share the parts.
template <typename T, uint32_t DP, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_attn_cache_join(const CacheArgs) {
    cargs& a = kernel_args();
    constexpr uint32_t U = 16;                                            // parts in flight
    const uint32_t lane = lane_id(), n32 = lane % 32u, hh = lane / 32u, wave = threadIdx.x / 64u;
    const uint32_t unit = uniform(quotient(blockIdx.x, a.per_block)), block = blockIdx.x - unit * a.blocks32;
    const uint32_t b = uniform(quotient(unit, a.per_kv)), head = unit - b * a.kv;
    const uint32_t f = SPLIT ? blockIdx.y : blockIdx.y * kWaves + wave, d = 8u * f + 4u * hh;
    if (8u * f >= a.dim) return;
    const Job job = {b, head, 0u, 0u, {}};
    const uint32_t rows = count_of(a, asked_of(a, b)) * a.group;
    if (block * kRows >= rows) return;
    const uint64_t first = part_index(a, b, head, block, 0);
    const Row row = row_of(a, job, block * kRows + n32, rows);
    const uint32_t per = SPLIT ? (a.parts + kWaves - 1u) / kWaves : a.parts;
    const uint32_t from = SPLIT ? wave * per : 0u, end = from + per < a.parts ? from + per : a.parts;
    f32x4 acc = (f32x4)(0.0f);
    float m = -INFINITY, l = 0.0f;
    // Sums of u in powers above the largest of all so far.
    auto add = [&](const auto& ml, const auto& x, auto n) {
        float next = m;
#pragma unroll
        for (uint32_t u = 0; u < decltype(n)::value; ++u) next = fmaxf(next, ml[u].x);
        const float at = next == -INFINITY ? 0.0f : next, fade = __builtin_amdgcn_exp2f(m - at);
        acc *= fade;
        l *= fade;
        m = next;
#pragma unroll
        for (uint32_t u = 0; u < decltype(n)::value; ++u) {
            if (ml[u].y == 0.0f) continue;                                // a part that saw no key left no sums
            const float w = __builtin_amdgcn_exp2f(ml[u].x - at);
            l += w * ml[u].y;
            acc += x[u] * w;
        }
    };
    if (row.valid) {
        for (uint32_t i0 = from; i0 < end; i0 += U) {
            float2 ml[U];
            f32x4 x[U];
#pragma unroll
            for (uint32_t u = 0; u < U; ++u) {
                ml[u] = make_float2(-INFINITY, 0.0f);
                x[u] = (f32x4)(0.0f);
                if (i0 + u >= end) continue;
                ml[u] = a.part_ml[(first + i0 + u) * 32u + n32];
                x[u] = part_at<DP>(a, first + i0 + u)[f * 64u + lane];
            }
            add(ml, x, std::integral_constant<uint32_t, U>{});
        }
    }
    if constexpr (SPLIT) {
        __shared__ float2 sums_ml[kWaves][64];
        __shared__ f32x4 sums[kWaves][64];
        sums_ml[wave][lane] = make_float2(m, l);
        sums[wave][lane] = acc;
        __syncthreads();
        if (wave) return;
        float2 ml[kWaves - 1];
        f32x4 x[kWaves - 1];
#pragma unroll
        for (uint32_t u = 1; u < kWaves; ++u) {
            ml[u - 1] = sums_ml[u][lane];
            x[u - 1] = sums[u][lane];
        }
        add(ml, x, std::integral_constant<uint32_t, kWaves - 1>{});
    }
    if (!row.valid) return;
    if (d < a.dim) store_result<T>(row, d, l == 0.0f ? (f32x4)(0.0f) : acc / l);
    if (f == 0 && hh == 0 && a.lse) store_lse(a, row, m, l);
}

// ---- host ---------------------------------------------------------------------------

// Shapes of the queries against a pool.
static bool shapes_fit(const View& q, const View& k) {
    return q.dim[0] == k.dim[0] && q.dim[0] % 8 == 0 && q.dim[0] <= 256 && q.dim[1] % k.dim[2] == 0 &&
           q.dim[1] <= 65535 && q.dim[2] <= 65535 && q.dim[3] <= 65535;
}

static uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }

// How the work is cut: fills the fields of `a` that follow from the shapes, the
// window and the hint alone and returns the workspace's bytes, 0 if there are
// more rows than 31 bits count or more workgroups than a launch holds.
static uint64_t plan(CacheArgs* a, uint32_t hint, bool codes) {
    constexpr uint64_t cus = 256;
    const uint32_t dp = padded_dim((uint32_t)a->q.dim[0]);
    a->dim = (uint32_t)a->q.dim[0];
    a->q_len = (uint32_t)a->q.dim[2];
    a->batch = (uint32_t)a->q.dim[3];
    a->kv = (uint32_t)a->k.dim[2];
    a->group = (uint32_t)a->q.dim[1] / a->kv;
    const uint64_t rows = (uint64_t)a->q_len * a->group;
    if (rows * a->batch > 0x7FFFFFFFull) return 0;
    a->per_group = 1.0 / a->group;
    const auto keys_of = [&](uint64_t block) -> uint64_t {                // keys of a block of rows: of the window, or all
        const uint64_t all = (uint64_t)a->window + a->sinks + ceil_div(block, a->group) + 1;
        return a->window && all < hint ? all : hint;
    };
    // Blocks of 32 rows, each with all of its keys, while all of them run at once and
    // their keys are few: the start is shorter (2 trees of 13 nodes x 4 heads of 700
    // tokens: 12.3 us, with shared tiles 14.1; 8 of 32 nodes of 2000 42 and 32, e4m3 35
    // and 47; 2048 queries of 2048 tokens, window 128: 59 and 24).
    const uint64_t shorts = (uint64_t)a->batch * a->kv * ceil_div(rows, kRows);
    const bool few = rows <= kRows || (shorts <= 2 * cus && shorts * keys_of(kRows) <= (codes ? 1u << 19 : 1u << 18));
    // Waves of a workgroup with many rows.  Eight share a tile's copies, and the work
    // of turning codes into elements (2048 queries of 32768 tokens: 972 us, with four
    // waves 1055; int8 beside f16 1234 and 1545, e4m3 1147 and 1329).  In 16 bits they
    // mask more where they see few keys (8192 queries, window 128: 98 and 88 us, window
    // 1024 200 and 197) and wait for each other where half of them have no rows (16 trees
    // of 120 rows: 75 and 69 us).  Codes cost more than that with any window (8192
    // queries, window 128: int8 124 and 134 us, e4m3 112 and 135; window 300: 5 x 777 queries
    // of 20 heads over 4 of 80 30 and 43, 777 of 40 over 8 of 128 30.7 and 31.6).
    // Above dim 128 a wave needs the registers of two; the twelve groups of a tile's copies
    // at dim 96 are no whole number for each of eight.
    const bool many = codes || (dp != 96 && rows > 4 * kRows && keys_of(8 * kRows) >= 2048);
    a->waves = few ? 0u : dp <= 128 && many ? 8u : 4u;
    const uint32_t waves = a->waves ? a->waves : 1u;
    const uint64_t keys = keys_of(kRows * waves);
    const uint64_t room = dp <= 128 && waves <= 4 ? 2 * cus : cus;         // workgroups that run at once
    a->blocks32 = (uint32_t)ceil_div(rows, kRows * waves) * waves;
    a->blocks = a->blocks32 / waves;
    const uint64_t jobs = (uint64_t)a->batch * a->kv * a->blocks;
    // Parts of 256 keys and above, of 128 while they leave compute units without one
    // (2 trees of 13 nodes of 700 tokens: 14.3 us, in parts of 256 15.7; 1 x 60 nodes of
    // 4000 tokens 27.9 and 23.9).  Few keys in one part: no second launch (512 keys of 64
    // elements 10.4 us, 12.3 in two parts; 128 rows with 400 keys 21.7 and 16.4; 777
    // queries, window 300, 40 heads: 20.5 in one part, 27.6 in two).
    uint64_t parts = 1;
    if (keys > (!a->waves ? 512u : a->window && jobs * a->waves > 256 ? 1024u : 256u)) {
        const auto least = [](uint64_t x, uint64_t y) { return x < y ? x : y; };
        const auto larger = [](uint64_t x, uint64_t y) { return x < y ? y : x; };
        parts = larger(least(ceil_div(keys, 256), room / jobs), least(ceil_div(keys, 128), cus / jobs));
        parts = larger(parts, 1);
        // Rounds of workgroups that are mostly full (40 sequences of 8192 tokens, 8 heads:
        // 228 us in one part, 198 in three).
        const auto full = [&](uint64_t n) { return (double)(jobs * n) / (double)(ceil_div(jobs * n, room) * room); };
        if (!a->waves && keys >= 2048)
            for (uint64_t n = parts + 1, end = parts + 3; n <= end; ++n)
                if (full(n) > 1.15 * full(parts)) parts = n;
    }
    a->parts = (uint32_t)parts;
    a->per_parts = 1.0 / a->parts;
    a->per_block = 1.0 / a->blocks32;
    a->per_kv = 1.0 / a->kv;
    a->direct = a->parts == 1;
    constexpr uint64_t most_groups = max_groups(kThreads);                 // of the products' launch, of the join's
    const uint64_t blocks = (uint64_t)a->batch * a->kv * a->blocks32;
    if (jobs * a->parts > most_groups || blocks > most_groups) return 0;
    const uint64_t pieces = a->direct ? 0 : blocks * a->parts;
    a->part_ml = reinterpret_cast<float2*>(pieces * dp * 32 * 4);          // behind the sums
    return pieces * (dp * 32 * 4 + 32 * 8) + 16;
}

template <typename T, uint32_t DP>
static void join(const CacheArgs& a, hipStream_t stream) {
    const uint32_t blocks = a.batch * a.kv * a.blocks32;
    // More parts than a wave has in flight: a workgroup's waves share them (a token of
    // 32768, 64 parts: both launches 48.5 us, so 39.6), or few blocks that leave the GPU
    // empty (a token of 4096 each of 4 rows 21.6 and 20.1; 2 trees of 60 nodes of 16000, 128
    // blocks, 54.8 and 56.6; 12 rows of 8192, 96 blocks, 71.5 and 72.6).
    if (a.parts > 16 || (a.parts > 4 && blocks <= 64))
        hipLaunchKernelGGL((k_attn_cache_join<T, DP, true>), dim3(blocks, (a.dim + 7u) / 8u), dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((k_attn_cache_join<T, DP, false>), dim3(blocks, (a.dim + 31u) / 32u), dim3(kThreads), 0, stream,
                           a);
}

template <typename T>
static tmap_status launch(const CacheArgs& a, int32_t format, hipStream_t stream, const char* name) {
    if (format == KV_SAME) launch_attn_cache<T, KV_SAME>(a, stream);
    else if (format == KV_INT8) launch_attn_cache<T, KV_INT8>(a, stream);
    else launch_attn_cache<T, KV_E4M3>(a, stream);
    const tmap_status st = check_launch(name);
    if (st || a.direct) return st;
    switch (padded_dim(a.dim)) {
    case 64: join<T, 64>(a, stream); break;
    case 96: join<T, 96>(a, stream); break;
    case 128: join<T, 128>(a, stream); break;
    case 192: join<T, 192>(a, stream); break;
    default: join<T, 256>(a, stream); break;
    }
    return check_launch(name);
}

static tmap_status attend(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, int32_t format,
                          const page_table_t* pt, const int32_t* d_rows, const int32_t* d_count, const int32_t* d_parent,
                          uint32_t window, uint32_t sinks, uint32_t len_hint, float scale, const tmap_t* o, float* d_lse,
                          void* d_ws, uint64_t ws_bytes, void* stream, const char* name) {
    if (!q || !k_pool || !v_pool || !pt || !o || !d_ws) return TMAP_ERR_NULL;
    CacheArgs a;
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
    if (format != KV_SAME && format != KV_INT8 && format != KV_E4M3) return TMAP_ERR_UNSUPPORTED;
    const int32_t tp = format == KV_SAME ? tq : (int32_t)TMAP_U8;
    const int64_t rows = format == KV_SAME ? pt->slots : code_rows(pt->slots, (uint64_t)a.k.dim[0]);
    if (tk != tp || tv != tp || to != tq || !same_dims(a.q, a.o) || !same_dims(a.k, a.v) || !shapes_fit(a.q, a.k) ||
        a.k.dim[1] != rows || (uint64_t)a.k.dim[3] != pt->pages || !std::isfinite(scale * kLog2e) ||
        (d_parent && a.q.dim[2] > kMaxNodes))
        return TMAP_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(d_ws) % 16 != 0) return TMAP_ERR_ALIGN;
    a.window = window;
    a.sinks = window ? sinks : 0;
    const uint64_t need = plan(&a, len_hint, format != KV_SAME);
    if (need == 0 || ws_bytes < need) return TMAP_ERR_UNSUPPORTED;
    a.part_o = static_cast<f32x4*>(d_ws);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(d_ws) + reinterpret_cast<uintptr_t>(a.part_ml));
    a.table = pt->d_table;
    a.lens = pt->d_lens;
    a.rows = d_rows;
    a.count = d_count;
    a.parent = d_parent;
    a.pitch = pt->pitch;
    a.table_rows = pt->rows;
    a.row_pages = pt->row_pages;
    a.pages = pt->pages;
    a.slots = pt->slots;
    a.per_slots = 1.0 / pt->slots;
    // Scores are kept in powers of two.  A negative scale turns the queries
    // around and a scale of 0 makes them 0, so that the factor is above 0 and
    // masked scores stay at -inf.
    a.zero = scale == 0;
    a.scale = a.zero ? 1.0f : std::fabs(scale) * kLog2e;
    a.flip = scale < 0 ? 0x80008000u : 0u;
    a.lse = d_lse;
    st = device_error_word(&a.err);
    if (st) return st;
    if (tq == TMAP_F16) return launch<_Float16>(a, format, as_stream(stream), name);
    return launch<__bf16>(a, format, as_stream(stream), name);
}

}  // namespace att

using namespace att;

extern "C" uint64_t attn_cache_workspace(const tmap_t* q, const tmap_t* k_pool, uint32_t window, uint32_t sinks,
                                         uint32_t len_hint) {
    CacheArgs a;
    std::memset(&a, 0, sizeof(a));
    int32_t tq, tk;
    if (view_of(q, 4, &a.q, &tq) || view_of(k_pool, 4, &a.k, &tk) || !shapes_fit(a.q, a.k)) return 0;
    a.window = window;
    a.sinks = window ? sinks : 0;
    return plan(&a, len_hint, tk == TMAP_U8);
}

extern "C" tmap_status attn_window(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, int32_t format,
                                   const page_table_t* pt, const int32_t* d_rows, const int32_t* d_count,
                                   uint32_t window, uint32_t sinks, uint32_t len_hint, float scale, const tmap_t* o,
                                   float* d_lse, void* d_ws, uint64_t ws_bytes, void* stream) {
    return attend(q, k_pool, v_pool, format, pt, d_rows, d_count, nullptr, window, sinks, len_hint, scale, o, d_lse,
                  d_ws, ws_bytes, stream, "attn_window");
}

extern "C" tmap_status attn_tree(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, int32_t format,
                                 const page_table_t* pt, const int32_t* d_rows, const int32_t* d_count,
                                 const int32_t* d_parent, uint32_t window, uint32_t sinks, uint32_t len_hint,
                                 float scale, const tmap_t* o, float* d_lse, void* d_ws, uint64_t ws_bytes,
                                 void* stream) {
    if (!d_parent) return TMAP_ERR_NULL;
    return attend(q, k_pool, v_pool, format, pt, d_rows, d_count, d_parent, window, sinks, len_hint, scale, o, d_lse,
                  d_ws, ws_bytes, stream, "attn_tree");
}
