// kernel_pages.hip -- the pages of the cache: handing out, sharing, giving
// back, copying and compacting.
//
// A page's use count says how many rows hold it.  Handing pages out takes a
// rank over the free pages (lowest index first) and a running sum over the
// entries that ask (in their order), so the result does not depend on timing.
// Both are taken by one workgroup: the counts of 64 Ki pages are read with all
// of its loads in flight, turned into one 64-bit word of busy bits per thread
// and ranked with population counts.  That is latency, not bandwidth: the
// tables of a cache are small beside its pages.  Moving pages is bandwidth:
// those kernels spread 16 KiB parts of pages over the whole GPU; compacting
// 16384 pages of 16 KiB in 8 pools, half of them in use, moves 1.07 GB in 202 us
// (5.3 TB/s) after 7.8 us for the plan; 500 pages copied within two pools take
// 10.8 us (6.1 TB/s, partly from the caches).  A small fork is its launches: free
// 2.6, hand out 5.3, rows and pages 4.4, extend 3.8 us.
#include <hip/hip_runtime.h>

#include <cstring>

#include "cache_util.hpp"

namespace att {

constexpr uint32_t kScanThreads = 1024;
constexpr uint32_t kSweep = 64u * kScanThreads;   // pages one sweep of the workgroup covers
constexpr uint32_t kCopyThreads = 256;
constexpr uint32_t kPartChunks = 4u * kCopyThreads;   // 16-byte chunks of one part of a page (16 KiB)
constexpr uint32_t kMaxPools = 256;
constexpr uint32_t kOnePages = 8192;              // pages that one launch compacts

struct Table {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    uint64_t pitch;
    uint32_t rows, row_pages, pages, slots;
};

static Table table_of(const page_table_t* pt) {
    return {pt->d_table, pt->d_lens, pt->d_refs, pt->pitch, pt->rows, pt->row_pages, pt->pages, pt->slots};
}

// The pools of one geometry: a page is n2 x n1 rows of row_bytes (dimensions
// that lie packed are merged, so a page without gaps is one row).
// Kernels take a few of them where that is enough: a launch costs the host
// 0.7 us more for each KiB of arguments.
template <uint32_t N>
struct PoolsOf {
    int64_t page;                 // bytes from one page to the next
    int64_t s1, s2;
    uint32_t npool, n1, n2;
    uint32_t row_bytes, row_chunks, chunks, parts;
    uint32_t magic_row, magic_n1; // multiply-high divisors, 0 for 1
    uint64_t base[N];
};
constexpr uint32_t kFewPools = 16;
typedef PoolsOf<kMaxPools> Pools;
typedef PoolsOf<kFewPools> FewPools;

static FewPools few(const Pools& p) {
    FewPools f;
    std::memcpy(&f, &p, sizeof(f));       // the same fields, fewer bases
    return f;
}

// ---- copying -------------------------------------------------------------------

// Division by an invariant for numerators below 2^24 (chunks of a page).
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t d, uint32_t magic) {
    const uint32_t q = fdiv(n, magic);
    return q * d > n ? q - 1 : q;
}

// One part (16 KiB) of one page, by 256 threads: the loads of a thread's four
// chunks are in flight together.  STREAM: the pages are many more than the
// caches hold, so neither side is kept there.
template <bool STREAM, uint32_t N>
__device__ __forceinline__ void copy_part(const PoolsOf<N>& p, uint32_t pool, int64_t from, int64_t to, uint32_t part,
                                          uint32_t thread) {
    const gbyte* src = gptr(p.base[pool]) + from * p.page;
    gbyte* dst = gptr(p.base[pool]) + to * p.page;
    u32x4 v[4];
    int64_t off[4];
    uint32_t left[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t c = part * kPartChunks + i * kCopyThreads + thread;
        left[i] = 0;
        if (c < p.chunks) {
            const uint32_t row = div_by(c, p.row_chunks, p.magic_row), k = c - row * p.row_chunks;
            const uint32_t r2 = div_by(row, p.n1, p.magic_n1);
            off[i] = (int64_t)r2 * p.s2 + (int64_t)(row - r2 * p.n1) * p.s1 + (int64_t)k * 16;
            left[i] = p.row_bytes - k * 16u;
            if (left[i] >= 16u)
                v[i] = STREAM ? __builtin_nontemporal_load((const ATT_GLOBAL u32x4*)(src + off[i]))
                              : *(const ATT_GLOBAL u32x4*)(src + off[i]);
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        if (left[i] >= 16u) {
            if (STREAM) __builtin_nontemporal_store(v[i], (ATT_GLOBAL u32x4*)(dst + off[i]));
            else *(ATT_GLOBAL u32x4*)(dst + off[i]) = v[i];
        } else for (uint32_t b = 0; b < left[i]; ++b) dst[off[i] + b] = src[off[i] + b];   // a row's last bytes
    }
}

template <uint32_t N>
__global__ __launch_bounds__(kCopyThreads) void k_page_copy(const PoolsOf<N> p, const int32_t* src, const int32_t* dst,
                                                            uint32_t pages, uint32_t* err) {
    const uint32_t i = blockIdx.x / p.parts, part = blockIdx.x - i * p.parts;
    const int32_t from = src[i], to = dst[i];
    if (from < 0 || to < 0) return;
    if ((uint32_t)from >= pages || (uint32_t)to >= pages) {
        if (threadIdx.x == 0) record_page_error(err);
        return;
    }
    copy_part<false>(p, blockIdx.y, from, to, part, threadIdx.x);
}

// ---- ranks ---------------------------------------------------------------------

// Exclusive sum of v over the workgroup's kScanThreads threads, and the total.
__device__ __forceinline__ uint32_t scan_block(uint32_t v, uint32_t* total) {
    __shared__ uint32_t part[kScanThreads / 64];
    const uint32_t lane = lane_id(), wave = threadIdx.x / 64u;
    uint32_t x = v;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();                     // the previous call's readers are done
    if (lane == 63) part[wave] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kScanThreads / 64; ++w) {
        const uint32_t s = part[w];
        before += w < wave ? s : 0u;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// Use counts of one sweep: thread t holds four pages of each 4096, so that
// reads are coalesced.  Pages past the last count as busy.
struct Counts {
    typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
    i32x4 v[16];
    __device__ __forceinline__ void load(const int32_t* refs, uint32_t base, uint32_t pages) {
#pragma unroll
        for (uint32_t u = 0; u < 16; ++u) {
            const uint32_t p = base + (u * kScanThreads + threadIdx.x) * 4u;
            v[u] = (i32x4)(1);
            if (base + u * kScanThreads * 4u >= pages) continue;         // the whole workgroup is past the end
            if (p + 4 <= pages) {
                v[u] = *(const ATT_GLOBAL i32x4*)(gptr(refs) + (uint64_t)p * 4u);
            } else {
                for (uint32_t k = 0; k < 4; ++k)
                    if (p + k < pages) v[u][k] = refs[p + k];
            }
        }
    }
    // Busy bits (count above 0) of the 64 pages from base + 64 * thread on: the
    // bits change hands in LDS.
    __device__ __forceinline__ uint64_t busy(uint32_t base, uint32_t pages) const {
        __shared__ uint8_t nibble[kSweep / 4];
        __syncthreads();                 // the previous sweep's readers are done
#pragma unroll
        for (uint32_t u = 0; u < 16; ++u) {
            if (base + u * kScanThreads * 4u >= pages) break;
            nibble[u * kScanThreads + threadIdx.x] =
                (uint8_t)((v[u][0] > 0) | (v[u][1] > 0) << 1 | (v[u][2] > 0) << 2 | (v[u][3] > 0) << 3);
        }
        __syncthreads();
        if (base + threadIdx.x * 64u >= pages) return ~0ull;
        uint64_t word = 0;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(nibble) + threadIdx.x * 4u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            uint32_t x = w[i];                           // four nibbles, one in each byte
            x = (x | x >> 4) & 0x00FF00FFu;
            x = (x | x >> 8) & 0xFFFFu;
            word |= (uint64_t)x << (16 * i);
        }
        return word;
    }
};

// ---- extend and fork -------------------------------------------------------------

// Workspace of extend and fork: for a fork the page each entry gets and the
// length its row starts from, and the free pages that do not fit into LDS.
struct AllocWs {
    int32_t* page;       // [n]: -1 none needed, -2 not served
    int32_t* held;       // [n]
    int32_t* fresh;      // [pages]
};
constexpr uint32_t kFreshLds = 4096;

// Entry i's need of pages, and the length of the row it starts from.  -1 for
// an entry that cannot be served.
template <bool FORK>
__device__ __forceinline__ int32_t entry_need(const Table& t, const int32_t* a, const int32_t* b, uint32_t i,
                                              int32_t* held, uint32_t* err) {
    *held = 0;
    const uint32_t src = (uint32_t)a[i];
    if (src >= t.rows) {
        record_page_error(err);
        return -1;
    }
    const int64_t len = t.lens[src], room = (int64_t)t.slots * t.row_pages;
    if (len < 0 || len > room) {
        record_page_error(err);
        return -1;
    }
    *held = (int32_t)len;
    if (FORK) {
        const uint32_t dst = (uint32_t)b[i];
        if (dst >= t.rows || t.lens[dst] != 0) {
            record_page_error(err);
            return -1;
        }
        return len % t.slots != 0;
    }
    const int64_t add = b[i];
    if (add < 0) {
        record_page_error(err);
        return -1;
    }
    if (len + add > room) return -1;
    return (int32_t)((uint32_t)(len + add + t.slots - 1) / t.slots - (uint32_t)(len + t.slots - 1) / t.slots);
}

// One workgroup hands out the lowest free pages.  Extend finishes here; fork
// leaves the rows and the data to k_fork_rows.  A chain of latencies (entries,
// their lengths, the counts, the stores), so the counts are on their way
// before the entries are looked at and nothing passes through memory between
// the steps: 16384 pages and 128 entries take 6.4 to 7.8 us, 1024 pages and 4
// entries 3.8 (extend) and 5.3 (fork).
template <bool FORK>
__global__ __launch_bounds__(kScanThreads) void k_hand_out(const Table t, const int32_t* a, const int32_t* b,
                                                           uint32_t n, int32_t* ok, AllocWs ws, uint32_t* err) {
    __shared__ int32_t fresh[kFreshLds];
    __shared__ uint64_t words[kScanThreads];
    __shared__ uint32_t ranks[kScanThreads];
    __shared__ uint32_t starts[kScanThreads + 1];
    __shared__ int32_t row_of[kScanThreads], first_of[kScanThreads];
    const uint32_t tid = threadIdx.x;
    Counts counts;
    counts.load(t.refs, 0, t.pages);
    // pages asked for by all entries; with one round of entries, each thread's stays in its registers
    int32_t held = 0, need = 0;
    uint32_t before = 0;
    uint64_t want = 0;
    for (uint32_t i0 = 0; i0 < n; i0 += kScanThreads) {
        const uint32_t i = i0 + tid;
        need = 0;
        if (i < n) need = entry_need<FORK>(t, a, b, i, &held, err);
        uint32_t all;
        before = scan_block(need > 0 ? (uint32_t)need : 0u, &all);       // a need is below 2^21
        want += all;
    }
    uint64_t found = 0;
    for (uint32_t base = 0; base < t.pages && found < want; base += kSweep) {
        if (base) counts.load(t.refs, base, t.pages);
        const uint64_t open = ~counts.busy(base, t.pages);
        uint32_t all;
        ranks[tid] = (uint32_t)found + scan_block((uint32_t)__popcll(open), &all);
        words[tid] = open;
        __syncthreads();
        for (uint32_t p = tid; p < kSweep; p += kScanThreads) {           // a thread for a page, as far as pages are wanted
            const uint32_t w = p / 64u, first = ranks[w];
            if (first >= want) break;
            const uint64_t bit = 1ull << (p % 64u);
            if (!(words[w] & bit)) continue;
            const uint32_t rank = first + (uint32_t)__popcll(words[w] & (bit - 1ull));
            if (rank >= want) break;
            if (rank < kFreshLds) fresh[rank] = (int32_t)(base + p);
            else ws.fresh[rank] = (int32_t)(base + p);
        }
        found += all;
    }
    // The list ends at the pages wanted, also where rows that are not distinct
    // come to need more of them further on.
    if (found > want) found = want;
    __syncthreads();                                      // the list is written, and every count was read
    auto page_at = [&](uint64_t rank) { return rank < kFreshLds ? fresh[rank] : ws.fresh[rank]; };
    uint64_t from = 0;                                    // pages of the entries of earlier rounds
    for (uint32_t i0 = 0; i0 < n; i0 += kScanThreads) {
        const uint32_t i = i0 + tid;
        uint32_t all = (uint32_t)want;
        if (n > kScanThreads) {
            need = 0;
            if (i < n) need = entry_need<FORK>(t, a, b, i, &held, err);
            before = scan_block(need > 0 ? (uint32_t)need : 0u, &all);
        }
        // An entry that needs no page is still served only while those before it are.
        const uint64_t start = from + before;
        const bool served = i < n && need >= 0 && start + (uint32_t)need <= found;
        if (i < n) ok[i] = served;
        if (FORK) {
            if (i < n) {
                const int32_t page = served && need ? page_at(start) : -1;
                if (page >= 0) t.refs[page] = 1;
                ws.page[i] = served ? page : -2;
                ws.held[i] = held;
            }
        } else {
            // the new pages: a thread for a page, which looks for its entry
            starts[tid] = before;
            row_of[tid] = served ? a[i] : -1;
            first_of[tid] = (int32_t)(((uint32_t)held + t.slots - 1u) / t.slots);
            if (tid == 0) starts[kScanThreads] = all;
            if (served) t.lens[(uint32_t)a[i]] = held + b[i];
            __syncthreads();
            for (uint32_t k = tid; k < all && from + k < found; k += kScanThreads) {
                uint32_t e = 0;                           // the last entry that starts at k or before
#pragma unroll
                for (uint32_t step = kScanThreads / 2; step; step /= 2)
                    if (starts[e + step] <= k) e += step;
                const int32_t row = row_of[e];
                if (row < 0) continue;
                const int32_t page = page_at(from + k);
                t.table[(uint64_t)(uint32_t)row * t.pitch + (uint32_t)first_of[e] + (k - starts[e])] = page;
                t.refs[page] = 1;
            }
            __syncthreads();
        }
        from += all;
    }
}

// Rows and data of a fork, after k_hand_out.  blockIdx.x: the entry; y (from
// first_y on): pieces of 1024 table entries first, then parts of the
// unfinished page, pool after pool.
template <uint32_t N>
__global__ __launch_bounds__(kCopyThreads) void k_fork_rows(const Table t, const PoolsOf<N> p, const int32_t* src,
                                                            const int32_t* dst, AllocWs ws, uint32_t pieces,
                                                            uint32_t first_y, uint32_t* err) {
    const uint32_t i = blockIdx.x, y = first_y + blockIdx.y;
    const int32_t fresh = ws.page[i];
    if (fresh == -2) return;
    const int32_t held = ws.held[i];
    const uint32_t full = (uint32_t)held / t.slots;
    const int32_t* from = t.table + (uint64_t)(uint32_t)src[i] * t.pitch;
    if (y < pieces) {
        int32_t* to = t.table + (uint64_t)(uint32_t)dst[i] * t.pitch;
        if (y == 0 && threadIdx.x == 0) t.lens[(uint32_t)dst[i]] = held;
        for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t c = y * 4u * kCopyThreads + k * kCopyThreads + threadIdx.x;
            if (c >= t.row_pages) break;
            int32_t page = -1;
            if (c < full) {
                page = from[c];
                if ((uint32_t)page < t.pages) atomicAdd(&t.refs[page], 1);
                else record_page_error(err);
            } else if (c == full) {
                page = fresh;
            }
            to[c] = page;
        }
        return;
    }
    if (fresh < 0) return;
    const uint32_t at = y - pieces, pool = at / p.parts, part = at - pool * p.parts;
    const int32_t last = from[full];
    if ((uint32_t)last >= t.pages) {
        if (threadIdx.x == 0 && at == 0) record_page_error(err);
        return;
    }
    copy_part<false>(p, pool, last, fresh, part, threadIdx.x);
}

// ---- free ------------------------------------------------------------------------

// blockIdx.x: the entry; y: pieces of 1024 table entries.  A page is taken
// out of the table with an exchange, so a row listed twice gives it back once.
__global__ __launch_bounds__(kCopyThreads) void k_page_free(const Table t, const int32_t* rows, uint32_t* err) {
    const uint32_t row = (uint32_t)rows[blockIdx.x];
    if (row >= t.rows) {
        if (threadIdx.x == 0) record_page_error(err);
        return;
    }
    int32_t* at = t.table + (uint64_t)row * t.pitch;
    if (blockIdx.y == 0 && threadIdx.x == 0) t.lens[row] = 0;
    for (uint32_t k = 0; k < 4; ++k) {
        const uint32_t c = blockIdx.y * 4u * kCopyThreads + k * kCopyThreads + threadIdx.x;
        if (c >= t.row_pages) break;
        if (at[c] == -1) continue;
        const int32_t page = atomicExch(&at[c], -1);
        if (page == -1) continue;
        if ((uint32_t)page < t.pages) atomicSub(&t.refs[page], 1);
        else record_page_error(err);
    }
}

// ---- compact ----------------------------------------------------------------------

struct CompactWs {
    uint64_t* busy;       // [words]: busy bits of 64 pages each
    uint32_t* before;     // [words]: busy pages before the word
    int32_t* hole;        // [pages]: free pages below U, ascending
    int32_t* mover;       // [pages]: busy pages at or above U, ascending
    uint32_t* count;      // U, how many move, busy pages below U
};

// Sweeps of 65536 pages: ranks first, then each thread lists the pages that
// it finds to be holes or movers.  With one sweep
// the words stay in LDS between the two.
__global__ __launch_bounds__(kScanThreads) void k_compact_plan(const Table t, CompactWs ws, int32_t* used) {
    __shared__ uint64_t words[kScanThreads];
    __shared__ uint32_t ranks[kScanThreads];
    __shared__ uint32_t below;                            // busy pages below U
    const uint32_t tid = threadIdx.x;
    const bool one = t.pages <= kSweep;
    Counts counts;
    uint32_t total = 0;
    for (uint32_t base = 0; base < t.pages; base += kSweep) {
        counts.load(t.refs, base, t.pages);
        uint64_t busy = counts.busy(base, t.pages);
        const uint32_t p = base + tid * 64u;
        // pages past the last are not in use here
        if (p + 64u > t.pages) busy &= p < t.pages ? (~0ull >> (p + 64u - t.pages)) : 0ull;
        uint32_t all;
        const uint32_t rank = total + scan_block((uint32_t)__popcll(busy), &all);
        if (p < t.pages) {
            ws.busy[p / 64u] = busy;
            ws.before[p / 64u] = rank;
        }
        words[tid] = busy;
        ranks[tid] = rank;
        total += all;
    }
    __syncthreads();                                      // the words are written
    const uint32_t U = total;
    auto word_of = [&](uint32_t w) { return one ? words[w] : ws.busy[w]; };
    auto rank_of = [&](uint32_t w) { return one ? ranks[w] : ws.before[w]; };
    if (tid == 0)
        below = U < t.pages ? rank_of(U / 64u) + (uint32_t)__popcll(word_of(U / 64u) & ((1ull << (U % 64u)) - 1ull)) : U;
    __syncthreads();
    const uint32_t kept = below;
    for (uint32_t p = tid; p < t.pages; p += kScanThreads) {
        const uint64_t word = word_of(p / 64u), bit = 1ull << (p % 64u);
        const bool busy = word & bit;
        if (busy == (p < U)) continue;                    // it stays as it is
        const uint32_t rank = rank_of(p / 64u) + (uint32_t)__popcll(word & (bit - 1ull));
        if (busy) ws.mover[rank - kept] = (int32_t)p;
        else ws.hole[p - rank] = (int32_t)p;
    }
    if (tid == 0) {
        ws.count[0] = U;
        ws.count[1] = U - kept;
        if (used) *used = (int32_t)U;
    }
}

// Where a page goes: itself below U, its rank's hole above, -1 if it is free there.
__device__ __forceinline__ int32_t new_place(const CompactWs& ws, uint32_t page, uint32_t U, uint32_t moves) {
    if (page < U) return (int32_t)page;
    const uint64_t word = ws.busy[page / 64u], bit = 1ull << (page % 64u);
    if (!(word & bit)) return -1;
    const uint32_t rank = ws.before[page / 64u] + (uint32_t)__popcll(word & (bit - 1ull));
    return ws.hole[rank - (U - moves)];
}

// Work items (mover, pool, part), the parts of a page side by side: 256 threads
// take items at, at + step, ...
template <uint32_t N>
__device__ __forceinline__ void move_pages(const PoolsOf<N>& p, uint32_t moves, const int32_t* mover,
                                           const int32_t* hole, uint32_t at, uint32_t step, uint32_t thread) {
    const uint32_t each = p.npool * p.parts;
    if (each == 0) return;
    const uint32_t step_m = step / each, step_r = step - step_m * each;
    uint32_t m = at / each, r = at - m * each;
    while (m < moves) {
        const uint32_t pool = r / p.parts;
        copy_part<true>(p, pool, mover[m], hole[m], r - pool * p.parts, thread);
        m += step_m;
        r += step_r;
        if (r >= each) {
            r -= each;
            ++m;
        }
    }
}

// The first table_blocks workgroups rewrite the table and the counts, the
// others move the pages.
template <uint32_t N>
__global__ __launch_bounds__(kCopyThreads) void k_compact_move(const Table t, int32_t* table_out, uint64_t pitch_out,
                                                               int32_t* refs_out, const PoolsOf<N> p, CompactWs ws,
                                                               uint32_t table_blocks, uint32_t* err) {
    const uint32_t U = ws.count[0], moves = ws.count[1];
    if (blockIdx.x < table_blocks) {
        const uint64_t step = (uint64_t)table_blocks * kCopyThreads, at = (uint64_t)blockIdx.x * kCopyThreads + threadIdx.x;
        for (uint64_t i = at; i < (uint64_t)t.rows * t.row_pages; i += step) {
            const uint32_t row = (uint32_t)(i / t.row_pages), c = (uint32_t)(i - (uint64_t)row * t.row_pages);
            int32_t page = t.table[(uint64_t)row * t.pitch + c];
            if (page >= 0) {
                if ((uint32_t)page < t.pages) page = new_place(ws, (uint32_t)page, U, moves);
                else record_page_error(err);
            }
            table_out[(uint64_t)row * pitch_out + c] = page;
        }
        for (uint64_t i = at; i < moves; i += step) {
            const int32_t h = ws.hole[i], m = ws.mover[i];
            const int32_t count = t.refs[m];
            refs_out[h] = count;
            refs_out[m] = 0;
        }
        if (refs_out != t.refs) {                         // the others keep theirs
            for (uint64_t i = at; i < t.pages; i += step) {
                const bool busy = ws.busy[i / 64u] >> (i % 64u) & 1u;
                if (busy == (i < U)) refs_out[i] = t.refs[i];
            }
        }
        return;
    }
    move_pages(p, moves, ws.mover, ws.hole, blockIdx.x - table_blocks, gridDim.x - table_blocks, threadIdx.x);
}

// Both in one launch, for a table of few pages that goes to memory of its own:
// each workgroup works the plan out for itself (nothing it reads is written),
// which costs less than a launch in between: 500 pages in two pools 8.2 us,
// 11.4 in two launches.  The lists of 8192 pages are what LDS holds beside the
// counts.
template <uint32_t N>
__global__ __launch_bounds__(kScanThreads) void k_compact_one(const Table t, int32_t* table_out, uint64_t pitch_out,
                                                              int32_t* refs_out, const PoolsOf<N> p, int32_t* used,
                                                              uint32_t* err) {
    __shared__ uint64_t words[kOnePages / 64];
    __shared__ uint32_t ranks[kOnePages / 64];
    __shared__ int32_t hole[kOnePages / 2], mover[kOnePages / 2];
    const uint32_t tid = threadIdx.x;
    Counts counts;
    counts.load(t.refs, 0, t.pages);
    uint64_t busy = counts.busy(0, t.pages);
    const uint32_t first = tid * 64u;
    if (first + 64u > t.pages) busy &= first < t.pages ? (~0ull >> (first + 64u - t.pages)) : 0ull;
    uint32_t U;
    const uint32_t rank0 = scan_block((uint32_t)__popcll(busy), &U);
    if (tid < kOnePages / 64u) {
        words[tid] = busy;
        ranks[tid] = rank0;
    }
    __syncthreads();
    auto rank_of = [&](uint32_t page) {                   // busy pages before it
        return ranks[page / 64u] + (uint32_t)__popcll(words[page / 64u] & ((1ull << (page % 64u)) - 1ull));
    };
    auto is_busy = [&](uint32_t page) { return (bool)(words[page / 64u] >> (page % 64u) & 1u); };
    const uint32_t kept = U < t.pages ? rank_of(U) : U, moves = U - kept;
    for (uint32_t i = tid; i < t.pages; i += kScanThreads) {
        if (is_busy(i) == (i < U)) continue;              // it stays as it is
        if (i < U) hole[i - rank_of(i)] = (int32_t)i;
        else mover[rank_of(i) - kept] = (int32_t)i;
    }
    __syncthreads();
    if (used && blockIdx.x == 0 && tid == 0) *used = (int32_t)U;
    const uint64_t step = (uint64_t)gridDim.x * kScanThreads, at = (uint64_t)blockIdx.x * kScanThreads + tid;
    for (uint64_t i = at; i < (uint64_t)t.rows * t.row_pages; i += step) {
        const uint32_t row = (uint32_t)(i / t.row_pages), c = (uint32_t)(i - (uint64_t)row * t.row_pages);
        int32_t page = t.table[(uint64_t)row * t.pitch + c];
        if (page >= (int32_t)U) {
            if ((uint32_t)page >= t.pages) record_page_error(err);
            else page = is_busy((uint32_t)page) ? hole[rank_of((uint32_t)page) - kept] : -1;
        }
        table_out[(uint64_t)row * pitch_out + c] = page;
    }
    for (uint64_t i = at; i < t.pages; i += step) {
        const uint32_t page = (uint32_t)i;
        const bool busy_now = is_busy(page);
        if (busy_now == (page < U)) refs_out[page] = t.refs[page];
        else refs_out[page] = busy_now ? 0 : t.refs[mover[page - rank_of(page)]];
    }
    constexpr uint32_t groups = kScanThreads / kCopyThreads;
    move_pages(p, moves, mover, hole, blockIdx.x * groups + tid / kCopyThreads, gridDim.x * groups, tid % kCopyThreads);
}

// ---- host ------------------------------------------------------------------------

static tmap_status pools_of(const tmap_t* maps, uint32_t npool, const page_table_t* pt, Pools* out, uint32_t* pages) {
    std::memset(out, 0, sizeof(*out));
    out->npool = npool;
    out->parts = 1;
    if (npool == 0) return TMAP_OK;
    if (!maps) return TMAP_ERR_NULL;
    if (npool > kMaxPools) return TMAP_ERR_UNSUPPORTED;
    View v;
    int32_t type = 0;
    for (uint32_t i = 0; i < npool; ++i) {
        View w;
        int32_t wt;
        const tmap_status st = view_of(maps + i, 4, &w, &wt);
        if (st) return st;
        if (i == 0) {
            v = w;
            type = wt;
        }
        if (wt != type || !same_dims(v, w)) return TMAP_ERR_UNSUPPORTED;
        for (int d = 0; d < 4; ++d)
            if (v.stride[d] != w.stride[d]) return TMAP_ERR_UNSUPPORTED;
        out->base[i] = w.base;
    }
    if (v.dim[3] > 0x7FFFFFFF) return TMAP_ERR_UNSUPPORTED;
    if (pt && ((uint64_t)v.dim[1] != pt->slots || (uint64_t)v.dim[3] != pt->pages)) return TMAP_ERR_UNSUPPORTED;
    // 256 MiB of one page; a map's dimensions may count more bytes than 64 bits
    constexpr uint64_t most = 1ull << 28;
    if ((unsigned __int128)v.dim[0] * v.stride[0] * v.dim[1] > most ||
        (unsigned __int128)v.dim[0] * v.stride[0] * v.dim[1] * v.dim[2] > most)
        return TMAP_ERR_UNSUPPORTED;
    uint64_t row = (uint64_t)v.dim[0] * (uint64_t)v.stride[0], n1 = (uint64_t)v.dim[1], n2 = (uint64_t)v.dim[2];
    int64_t s1 = v.stride[1], s2 = v.stride[2];
    if (s2 < s1 || n1 == 1) {                             // the closer dimension first
        const int64_t s = s1;
        const uint64_t n = n1;
        s1 = s2, n1 = n2, s2 = s, n2 = n;
    }
    if (n1 == 1 || (uint64_t)s1 == row) {
        row *= n1;
        n1 = n2, s1 = s2, n2 = 1, s2 = 0;
        if (n1 == 1 || (uint64_t)s1 == row) {
            row *= n1;
            n1 = 1, s1 = 0;
        }
    }
    const uint64_t row_chunks = (row + 15) / 16, chunks = row_chunks * n1 * n2;
    if (chunks > most / 16) return TMAP_ERR_UNSUPPORTED;      // rows are copied in whole chunks
    out->page = v.stride[3];
    out->s1 = s1;
    out->s2 = s2;
    out->n1 = (uint32_t)n1;
    out->n2 = (uint32_t)n2;
    out->row_bytes = (uint32_t)row;
    out->row_chunks = (uint32_t)row_chunks;
    out->chunks = (uint32_t)chunks;
    out->parts = (uint32_t)((chunks + kPartChunks - 1) / kPartChunks);
    out->magic_row = magic_for(out->row_chunks);
    out->magic_n1 = magic_for(out->n1);
    *pages = (uint32_t)v.dim[3];
    return TMAP_OK;
}

static uint64_t align16(uint64_t x) { return (x + 15) & ~15ull; }

static uint64_t alloc_bytes(uint32_t pages, uint32_t n) { return 2 * align16(4ull * n) + align16(4ull * pages); }

static AllocWs alloc_ws(void* ws, uint32_t n) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    const uint64_t list = align16(4ull * n);
    return {(int32_t*)p, (int32_t*)(p + list), (int32_t*)(p + 2 * list)};
}

static uint64_t compact_bytes(uint32_t pages) {
    const uint64_t words = ((uint64_t)pages + 63) / 64;
    return align16(8 * words) + align16(4 * words) + 2 * align16(4ull * pages) + 16;
}

static CompactWs compact_ws(void* ws, uint32_t pages) {
    const uint64_t words = ((uint64_t)pages + 63) / 64;
    uint8_t* p = static_cast<uint8_t*>(ws);
    CompactWs w;
    w.busy = (uint64_t*)p;
    p += align16(8 * words);
    w.before = (uint32_t*)p;
    p += align16(4 * words);
    w.hole = (int32_t*)p;
    p += align16(4ull * pages);
    w.mover = (int32_t*)p;
    p += align16(4ull * pages);
    w.count = (uint32_t*)p;
    return w;
}

static tmap_status check_ws(const void* ws, uint64_t bytes, uint64_t need) {
    if (!ws) return TMAP_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return TMAP_ERR_ALIGN;
    return bytes < need ? TMAP_ERR_UNSUPPORTED : TMAP_OK;
}

}  // namespace att

using namespace att;

extern "C" uint64_t page_workspace(const page_table_t* pt, uint32_t n) {
    if (!pt) return 0;
    const uint64_t a = alloc_bytes(pt->pages, n), c = compact_bytes(pt->pages);
    return a > c ? a : c;
}

extern "C" tmap_status page_copy(const tmap_t* pools, uint32_t npool, const int32_t* d_src, const int32_t* d_dst,
                                 uint32_t n, void* stream) {
    if (!pools) return TMAP_ERR_NULL;
    if (npool == 0) return TMAP_ERR_UNSUPPORTED;
    Pools p;
    uint32_t pages = 0;
    tmap_status st = pools_of(pools, npool, nullptr, &p, &pages);
    if (st) return st;
    if (n == 0) return TMAP_OK;
    if (!d_src || !d_dst) return TMAP_ERR_NULL;
    uint32_t* err = nullptr;
    st = device_error_word(&err);
    if (st) return st;
    const dim3 block(kCopyThreads);
    const hipStream_t s = as_stream(stream);
    const uint32_t most = max_groups(kCopyThreads) / p.parts;              // entries of a launch
    for (uint32_t i = 0, m = 0; i < n; i += m) {
        m = n - i < most ? n - i : most;
        const dim3 grid(m * p.parts, npool);
        if (npool <= kFewPools)
            hipLaunchKernelGGL(k_page_copy, grid, block, 0, s, few(p), d_src + i, d_dst + i, pages, err);
        else hipLaunchKernelGGL(k_page_copy, grid, block, 0, s, p, d_src + i, d_dst + i, pages, err);
    }
    return check_launch("page_copy");
}

extern "C" tmap_status page_extend(const page_table_t* pt, const int32_t* d_rows, const int32_t* d_add, uint32_t n,
                                   int32_t* d_ok, void* d_ws, uint64_t ws_bytes, void* stream) {
    tmap_status st = check_table(pt);
    if (st) return st;
    if (!pt->d_lens || !pt->d_refs) return TMAP_ERR_NULL;
    if (n == 0) return TMAP_OK;
    if (!d_rows || !d_add || !d_ok) return TMAP_ERR_NULL;
    if (n > 0x7FFFFFFFu) return TMAP_ERR_UNSUPPORTED;      // the kernel counts them in steps of its threads
    st = check_ws(d_ws, ws_bytes, alloc_bytes(pt->pages, n));
    if (st) return st;
    uint32_t* err = nullptr;
    st = device_error_word(&err);
    if (st) return st;
    hipLaunchKernelGGL(k_hand_out<false>, dim3(1), dim3(kScanThreads), 0, as_stream(stream), table_of(pt), d_rows,
                       d_add, n, d_ok, alloc_ws(d_ws, n), err);
    return check_launch("page_extend");
}

extern "C" tmap_status page_fork(const page_table_t* pt, const tmap_t* pools, uint32_t npool, const int32_t* d_src,
                                 const int32_t* d_dst, uint32_t n, int32_t* d_ok, void* d_ws, uint64_t ws_bytes,
                                 void* stream) {
    tmap_status st = check_table(pt);
    if (st) return st;
    if (!pt->d_lens || !pt->d_refs) return TMAP_ERR_NULL;
    Pools p;
    uint32_t pages = 0;
    st = pools_of(pools, npool, pt, &p, &pages);
    if (st) return st;
    if (n == 0) return TMAP_OK;
    if (!d_src || !d_dst || !d_ok) return TMAP_ERR_NULL;
    st = check_ws(d_ws, ws_bytes, alloc_bytes(pt->pages, n));
    if (st) return st;
    const uint32_t pieces = (pt->row_pages + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
    const uint32_t all_y = pieces + npool * p.parts;
    if (n > 0x7FFFFFFFu) return TMAP_ERR_UNSUPPORTED;
    uint32_t* err = nullptr;
    st = device_error_word(&err);
    if (st) return st;
    AllocWs ws = alloc_ws(d_ws, n);
    const hipStream_t s = as_stream(stream);
    hipLaunchKernelGGL(k_hand_out<true>, dim3(1), dim3(kScanThreads), 0, s, table_of(pt), d_src, d_dst, n, d_ok, ws,
                       err);
    st = check_launch("page_fork");
    if (st) return st;
    constexpr uint32_t most = max_groups(kCopyThreads), most_y = 65535;
    const dim3 block(kCopyThreads);
    for (uint32_t i = 0, m = 0; i < n; i += m, ws.page += m, ws.held += m) {
        m = n - i < most ? n - i : most;
        for (uint32_t y = 0; y < all_y; y += most_y) {
            const dim3 grid(m, all_y - y < most_y ? all_y - y : most_y);
            if (npool <= kFewPools)
                hipLaunchKernelGGL(k_fork_rows, grid, block, 0, s, table_of(pt), few(p), d_src + i, d_dst + i, ws,
                                   pieces, y, err);
            else
                hipLaunchKernelGGL(k_fork_rows, grid, block, 0, s, table_of(pt), p, d_src + i, d_dst + i, ws, pieces,
                                   y, err);
        }
    }
    return check_launch("page_fork");
}

extern "C" tmap_status page_free(const page_table_t* pt, const int32_t* d_rows, uint32_t n, void* stream) {
    tmap_status st = check_table(pt);
    if (st) return st;
    if (!pt->d_lens || !pt->d_refs) return TMAP_ERR_NULL;
    if (n == 0) return TMAP_OK;
    if (!d_rows) return TMAP_ERR_NULL;
    const uint32_t pieces = (pt->row_pages + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
    uint32_t* err = nullptr;
    st = device_error_word(&err);
    if (st) return st;
    constexpr uint32_t most = max_groups(kCopyThreads);
    for (uint32_t i = 0, m = 0; i < n; i += m) {
        m = n - i < most ? n - i : most;
        hipLaunchKernelGGL(k_page_free, dim3(m, pieces), dim3(kCopyThreads), 0, as_stream(stream), table_of(pt),
                           d_rows + i, err);
    }
    return check_launch("page_free");
}

extern "C" tmap_status page_compact(const page_table_t* from, const page_table_t* to, const tmap_t* pools,
                                    uint32_t npool, int32_t* d_used, void* d_ws, uint64_t ws_bytes, void* stream) {
    tmap_status st = check_table(from);
    if (st == TMAP_OK) st = check_table(to);
    if (st) return st;
    if (!from->d_refs || !to->d_refs) return TMAP_ERR_NULL;
    if (from->rows != to->rows || from->row_pages != to->row_pages || from->pages != to->pages ||
        from->slots != to->slots)
        return TMAP_ERR_UNSUPPORTED;
    if (from->d_table == to->d_table && from->pitch != to->pitch) return TMAP_ERR_UNSUPPORTED;
    Pools p;
    uint32_t pages = 0;
    st = pools_of(pools, npool, from, &p, &pages);
    if (st) return st;
    st = check_ws(d_ws, ws_bytes, compact_bytes(from->pages));
    if (st) return st;
    uint32_t* err = nullptr;
    st = device_error_word(&err);
    if (st) return st;
    uint32_t cus = 0;
    st = device_cu_count(&cus);
    if (st) return st;
    const hipStream_t s = as_stream(stream);
    const uint64_t most = ((uint64_t)from->pages / 2) * npool * p.parts;   // parts of pages that could move
    if (from->pages <= kOnePages && from->d_table != to->d_table && from->d_refs != to->d_refs) {
        constexpr uint64_t groups = kScanThreads / kCopyThreads;
        const uint64_t rewrite = ((uint64_t)from->rows * from->row_pages + 4 * kScanThreads - 1) / (4 * kScanThreads);
        const uint64_t want = (most + groups - 1) / groups > rewrite ? (most + groups - 1) / groups : rewrite;
        const dim3 grid((uint32_t)(want < 2ull * cus ? want : 2ull * cus)), block(kScanThreads);
        if (npool <= kFewPools)
            hipLaunchKernelGGL(k_compact_one, grid, block, 0, s, table_of(from), to->d_table, to->pitch, to->d_refs,
                               few(p), d_used, err);
        else
            hipLaunchKernelGGL(k_compact_one, grid, block, 0, s, table_of(from), to->d_table, to->pitch, to->d_refs, p,
                               d_used, err);
        return check_launch("page_compact");
    }
    const CompactWs ws = compact_ws(d_ws, from->pages);
    hipLaunchKernelGGL(k_compact_plan, dim3(1), dim3(kScanThreads), 0, as_stream(stream), table_of(from), ws, d_used);
    st = check_launch("page_compact");
    if (st) return st;
    // how many pages move is known on the device alone: as many workgroups as keep the GPU full, at most one for
    // each part that could move (half of the pages)
    const uint64_t entries = (uint64_t)from->rows * from->row_pages + from->pages;
    const uint64_t tb = (entries + 4 * kCopyThreads - 1) / (4 * kCopyThreads);
    const uint32_t table_blocks = (uint32_t)(tb < 4ull * cus ? tb : 4ull * cus);
    const uint32_t movers = (uint32_t)(most < 8ull * cus ? most : 8ull * cus);
    const dim3 grid(table_blocks + movers), block(kCopyThreads);
    if (npool <= kFewPools)
        hipLaunchKernelGGL(k_compact_move, grid, block, 0, s, table_of(from), to->d_table, to->pitch, to->d_refs,
                           few(p), ws, table_blocks, err);
    else
        hipLaunchKernelGGL(k_compact_move, grid, block, 0, s, table_of(from), to->d_table, to->pitch, to->d_refs, p,
                           ws, table_blocks, err);
    return check_launch("page_compact");
}
