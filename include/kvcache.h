/*
 * kvcache.h -- C ABI of a paged key / value cache on MI355X (gfx950): rotary
 * positions, the pages, pools of 8 bits an element, and attention: behind a
 * shared prefix, with a sliding window, and of a tree of drafted tokens.
 *
 * Keys and values live in pools of pages.  A pool is described by a tensor
 * map (tmap.h) of rank 4 with dims {dim, slots, heads, pages}: page p holds
 * `slots` tokens of `heads` heads of `dim` elements, in whatever order the
 * map's strides say.  Of a map these calls read the base, the dimensions,
 * the strides and the element type; box, element strides (which must be 1),
 * swizzle and fill play no part.
 *
 * The conventions of tmap.h hold: dimensions innermost first, d_ pointers
 * are device addresses, launches are asynchronous on `stream` and can be
 * captured into a graph, nothing is allocated, and errors are returned.
 * What a kernel finds wrong in device memory (a row, position or page out of
 * range) it skips: nothing out of range is read or written, the calls' own
 * outputs say so where they are documented to, and the event is recorded for
 * tile_device_status (TMAP_ERR_PAGE).
 */
#ifndef ATT_KVCACHE_H
#define ATT_KVCACHE_H

#include "tmap.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the page table ---------------------------------------------------------- */

/* Device memory that says which pages hold which sequence.  Row r is one
 * sequence: its token t lies in page d_table[r * pitch + t / slots], slot
 * t % slots.  Unused entries are -1.  A shared prefix is a row like any
 * other.  The struct itself is read on the host before a call returns. */
typedef struct {
    int32_t* d_table;      /* rows x row_pages page numbers                       */
    int32_t* d_lens;       /* tokens each row holds, [rows]                       */
    int32_t* d_refs;       /* rows that use each page, [pages]; <= 0 is free      */
    uint64_t pitch;        /* entries from one row to the next, >= row_pages      */
    uint32_t rows;
    uint32_t row_pages;    /* entries a row can use, below 2^21                   */
    uint32_t pages;        /* pages of the pools, at most 2^31 - 1                */
    uint32_t slots;        /* tokens per page, at least 1; slots * row_pages is
                              at most 2^31 - 1                                    */
} page_table_t;

/* ---- rotary positions -------------------------------------------------------- */

/* Opaque plan of a rotation, created on the host and copyable by value. */
typedef struct rope_t {
    uint8_t opaque[1072];
} __attribute__((aligned(16))) rope_t;

enum { ROPE_HALF = 0, ROPE_INTERLEAVED = 1 };
enum { ROPE_SCALE_NONE = 0, ROPE_SCALE_LINEAR = 1, ROPE_SCALE_BASE = 2, ROPE_SCALE_RAMP = 3 };

/* Encode a rotation of the first rot_dim elements of each head (even, 2 to
 * 256).  Pair j of rot_dim / 2 consists of elements (j, j + rot_dim / 2)
 * (ROPE_HALF) or (2j, 2j + 1) (ROPE_INTERLEAVED) and turns by
 * position * theta_j:
 *   first'  = magnitude * (first * cos - second * sin)
 *   second' = magnitude * (first * sin + second * cos)
 * with theta_j = base^(-2j / rot_dim), or, for contexts longer than the
 * trained one:
 *   LINEAR  theta_j / factor
 *   BASE    the base replaced by base * factor^(rot_dim / (rot_dim - 2))
 *           (rot_dim = 2 has only theta_0 = 1)
 *   RAMP    theta_j * (w + (1 - w) / factor), w = (n_j - slow) / (fast - slow)
 *           clamped to [0, 1], n_j = original_len * theta_j / 2 pi the turns
 *           of pair j over the trained context.
 * Angles are kept in 64 bits, the magnitude in 32.  Errors: NULL; UNSUPPORTED
 * (enum, rot_dim, base or factor not above 0, magnitude not finite in fp32, a
 * base or an angle that is not finite in 64 bits, for RAMP original_len 0 or
 * fast <= slow). */
tmap_status rope_encode(rope_t* out, uint32_t rot_dim, int32_t layout, double base, int32_t scaling, double factor,
                        uint32_t original_len, double slow, double fast, double magnitude);

/* y = x rotated: token t of x (map dims {dim, heads, tokens}) turns by
 * d_pos[t], any int32; elements past rot_dim are copied.  y has x's type and
 * dims and may be x itself (any other overlap is not allowed).  inverse != 0
 * turns by the negative angle, magnitude kept: the gradient of the forward
 * call.  Types f16, bf16, f32; the angle is reduced in 64 bits, the rotation
 * is computed in fp32 and rounded once.  Errors: NULL, DTYPE, RANK,
 * UNSUPPORTED (im2col map, element strides, dims differ, dim < rot_dim,
 * dim > 256, more than 2^31 - 1 tokens or 65535 heads), HIP. */
tmap_status rope_apply(const rope_t* r, const tmap_t* x, const tmap_t* y, const int32_t* d_pos, int32_t inverse,
                       void* stream);

/* One step's tokens: q_out = q rotated (both NULL: no queries), k rotated and
 * v as it is written to the cache.  q, k and v have dims {dim, heads,
 * tokens}, k and v as many heads as the pools.  Token t turns by d_pos[t] and
 * goes to row d_rows[t], token index d_at[t] of the row; a negative d_rows[t]
 * writes no key and value (padding).  The pages have to be in the table
 * already (page_extend); r == NULL writes the keys unrotated and needs no
 * d_pos.  Of pt only the table is read.  Two tokens for one slot race.
 * Errors as rope_apply, plus UNSUPPORTED where pools, table and tensors do
 * not fit each other. */
tmap_status rope_append(const rope_t* r, const tmap_t* q, const tmap_t* q_out, const tmap_t* k, const tmap_t* v,
                        const tmap_t* k_pool, const tmap_t* v_pool, const page_table_t* pt, const int32_t* d_rows,
                        const int32_t* d_at, const int32_t* d_pos, void* stream);

/* ---- pools of 8 bits an element ------------------------------------------------ */

/* What a pool's elements are: of the queries' type, or 8-bit codes c that
 * stand for c * s, with a scale s for each token and head.  A pool of codes is
 * a map of type u8 with dims {dim, kv8_rows(slots, dim), heads, pages}, dim a
 * multiple of 16: in each head of a page the slots' codes are followed by the
 * slots' scales, bf16 side by side, that of slot i at row slots + 2i / dim,
 * byte 2i % dim.  page_copy, page_fork, page_compact and page_keep take such
 * pools like any others. */
enum { KV_SAME = 0, KV_INT8 = 1, KV_E4M3 = 2 };

/* Rows of dim bytes that a head of a page with `slots` tokens takes, codes and
 * scales (0 for a dim that is no multiple of 16 or above 256, or no slots). */
uint32_t kv8_rows(uint32_t slots, uint32_t dim);

/* rope_append to pools of codes.  With y the rotated key (or the value) of a
 * head in fp32, and Z the largest code, 127 or 448: s is max |y| / Z rounded up
 * to bf16, and c is y / s rounded to the nearest code, ties to even (0 where s
 * is 0).  A head that holds an infinity or a NaN gets the scale NaN: it reads
 * as NaN.  Types f16 and bf16; everything else, q_out among it, as
 * rope_append.  Errors as rope_append, and UNSUPPORTED for another format. */
tmap_status kv8_append(const rope_t* r, const tmap_t* q, const tmap_t* q_out, const tmap_t* k, const tmap_t* v,
                       int32_t format, const tmap_t* k_pool, const tmap_t* v_pool, const page_table_t* pt,
                       const int32_t* d_rows, const int32_t* d_at, const int32_t* d_pos, void* stream);

/* Tokens of pools of codes read back: token t of k and v (dims {dim, heads,
 * tokens}, types f16, bf16, f32) is token d_at[t] of row d_rows[t], c * s
 * rounded once to the type.  Where d_rows[t] is negative, or there is no such
 * token's page, k and v stay as they were.  Of pt only the table is read.
 * Errors as kv8_append. */
tmap_status kv8_read(int32_t format, const tmap_t* k_pool, const tmap_t* v_pool, const page_table_t* pt,
                     const int32_t* d_rows, const int32_t* d_at, const tmap_t* k, const tmap_t* v, void* stream);

/* ---- pages ------------------------------------------------------------------- */

/* Bytes of workspace that page_fork and page_extend with up to n entries, and
 * page_compact, need for this table (0 for a NULL table).  A workspace may be
 * reused by the next call on the same stream; its contents mean nothing. */
uint64_t page_workspace(const page_table_t* pt, uint32_t n);

/* Copy page d_src[i] to page d_dst[i] for i < n, in each of npool pools (1 to
 * 256, all of one geometry: type, dims, strides; e.g. every layer's keys and
 * values).  An entry with a negative page number is skipped.  A page that is
 * both written and read, or written twice, races.  Errors: NULL, RANK,
 * UNSUPPORTED (pools, or a page of more than 256 MiB, its rows counted in whole
 * 16 bytes), HIP.  n == 0 is a no-op. */
tmap_status page_copy(const tmap_t* pools, uint32_t npool, const int32_t* d_src, const int32_t* d_dst, uint32_t n,
                      void* stream);

/* Row d_rows[i] grows by d_add[i] >= 0 tokens, i < n; pages it lacks are the
 * free ones of lowest index, handed out in the order of i.  Entry i is served
 * (d_ok[i] = 1) while the pages that entries 0..i need together are free;
 * from the first that does not fit on, entries are left as they were
 * (d_ok[i] = 0).  So is an entry whose row cannot hold the tokens (it needs
 * no pages).  Rows are distinct.  Errors: NULL, UNSUPPORTED (table, workspace
 * too small, n above 2^31 - 1), ALIGN (workspace not 16-byte aligned), HIP.
 * n == 0 is a no-op. */
tmap_status page_extend(const page_table_t* pt, const int32_t* d_rows, const int32_t* d_add, uint32_t n,
                        int32_t* d_ok, void* d_ws, uint64_t ws_bytes, void* stream);

/* Row d_dst[i] becomes a copy of row d_src[i], i < n: full pages are shared
 * (their counts go up by one), an unfinished last page gets a page of its
 * own, the free one of lowest index in the order of i, and is copied in every
 * pool.  d_ok and shortage as page_extend (a row that is not served stays
 * empty).  Destination rows are empty (page_free) and distinct; a row that
 * holds tokens is not served.  pools may be NULL with npool == 0: the tables
 * alone.  Errors as page_extend and page_copy. */
tmap_status page_fork(const page_table_t* pt, const tmap_t* pools, uint32_t npool, const int32_t* d_src,
                      const int32_t* d_dst, uint32_t n, int32_t* d_ok, void* d_ws, uint64_t ws_bytes, void* stream);

/* Rows d_rows[i], i < n, give their pages back: counts go down by one, table
 * entries become -1, lengths 0.  A row that is listed twice, or is empty,
 * gives back what it holds once.  Errors: NULL, UNSUPPORTED (table), HIP. */
tmap_status page_free(const page_table_t* pt, const int32_t* d_rows, uint32_t n, void* stream);

/* Move the U pages in use (count above 0) to indices below U: the i-th used
 * page at or above U goes to the i-th free page below U, both in ascending
 * order.  `to` receives the table and the counts (its d_lens is not used): it
 * has from's sizes, and is `from` itself or does not overlap it; with a table
 * of its own the old one still reads the old pages, which keep their
 * contents, so steps in flight may go on using it.  Every one of the
 * rows x row_pages entries is rewritten, one that names a free page at or
 * above U as -1.  *d_used (may be NULL) receives U.  Errors as page_fork. */
tmap_status page_compact(const page_table_t* from, const page_table_t* to, const tmap_t* pools, uint32_t npool,
                         int32_t* d_used, void* d_ws, uint64_t ws_bytes, void* stream);

/* The tokens of row d_rows[i] from index d_from[i] on are replaced by some of
 * them, i < n: token d_from[i] + d_keep[i * width + j] becomes token d_from[i] +
 * j for j < d_count[i], in every pool, and the row then ends; the pages between
 * its new end and the old one are given back.  So a row keeps the accepted ones
 * of its drafted tokens.
 * The d_count[i] <= width kept indices ascend from 0 or above and end below the
 * row's length (none: the row is cut to d_from[i]).  d_ok[i] = 1, or 0 for an
 * entry that is left as it was: where that does not hold, where a page that
 * would be written is shared (count above 1), or where the row would come to
 * end inside of a shared page, which it would write as it grows again (fork it).
 * Rows are distinct (of one that is listed twice every page is given back once).
 * pools may be NULL with npool == 0: the tables alone.  Errors: NULL, RANK,
 * UNSUPPORTED (table, pools), HIP.  n == 0 is a no-op. */
tmap_status page_keep(const page_table_t* pt, const tmap_t* pools, uint32_t npool, const int32_t* d_rows,
                      const int32_t* d_from, const int32_t* d_keep, uint32_t width, const int32_t* d_count, uint32_t n,
                      int32_t* d_ok, void* stream);

/* ---- attention ---------------------------------------------------------------- */

/* Bytes of workspace that attn_shared_prefix needs for these queries, this
 * pool, prefix_len and suffix_hint (0 if they are not valid). */
uint64_t attn_workspace(const tmap_t* q, const tmap_t* k_pool, uint32_t prefix_len, uint32_t suffix_hint);

/* Attention of a batch whose sequences share their first prefix_len tokens.
 * q and o have dims {dim, heads, q_len, batch}; query j of sequence b sees
 * the prefix (the first prefix_len tokens of table row prefix_row; the row is
 * not read when prefix_len is 0) and of its own row r = d_rows[b] (NULL: b)
 * the first d_lens[r] - q_len + 1 + j tokens: its own key is the last it
 * sees.  The prefix is read once for the whole batch.
 *   o   = sum_t softmax_t(scale * q . k_t) v_t
 *   lse = log sum_t exp(scale * q . k_t), fp32 [batch, q_len, heads] (NULL:
 *         not written)
 * A query that sees nothing, or whose scores are all -inf, gets o = 0 and
 * lse = -inf; a NaN or +inf among its scores makes both NaN.  Query head h uses
 * key / value head h / (heads / kv heads).  Keys and values that a query does
 * not see do not reach it, whatever they hold.  Lengths are read on the
 * device, so that a captured call follows them; suffix_hint is the length
 * that the work is split for (any value is right).  Types f16 and bf16;
 * scores, statistics and sums are fp32, the weights are rounded to the
 * element type for the product with the values.  dim is a multiple of 8, at
 * most 256.  Errors: NULL, DTYPE, RANK, ALIGN (workspace), UNSUPPORTED
 * (shapes, heads not a multiple of the pool's, prefix_row, prefix_len beyond
 * the row, scale * log2(e) not finite in fp32, workspace too small, heads,
 * q_len or batch above 65535, more than 2^31 - 1 queries for a key / value
 * head, more than 2^24 - 1 workgroups: about one for each sequence, key / value
 * head and 32 of its queries), HIP.  An empty batch is not expressible (a map's
 * dimensions are at least 1). */
tmap_status attn_shared_prefix(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, const page_table_t* pt,
                               uint32_t prefix_row, uint32_t prefix_len, const int32_t* d_rows, uint32_t suffix_hint,
                               float scale, const tmap_t* o, float* d_lse, void* d_ws, uint64_t ws_bytes,
                               void* stream);

/* Bytes of workspace that attn_window and attn_tree need for these queries,
 * this pool, window, sinks and len_hint (0 if they are not valid). */
uint64_t attn_cache_workspace(const tmap_t* q, const tmap_t* k_pool, uint32_t window, uint32_t sinks,
                              uint32_t len_hint);

/* Causal attention of sequences over the cache.  q and o have dims {dim, heads,
 * q_len, batch}; of sequence b the first n = d_count[b] queries (NULL: q_len)
 * are there, and what o and d_lse hold for the others stays as it was.  Its
 * tokens are those of row r = d_rows[b] (NULL: b), and its queries the last n of
 * them: query j stands at p = d_lens[r] - n + j and sees the tokens t <= p that
 * are within the window, t > p - window, or among the first `sinks` ones
 * (window 0: every t <= p).  o, lse, heads, types, scale and the rounding as
 * attn_shared_prefix, but that an f16 weight vanishes below 2^-32 of the largest
 * (there below 2^-25); a query that sees nothing gets o = 0 and lse = -inf, and
 * what a query does not see does not reach it, whatever it holds.  The pools are
 * of the queries' type (KV_SAME) or hold codes; a key is c * s, and so is a value
 * (f16: where c times the power of two in s is beyond the type's numbers it is an
 * infinity, and below its normal numbers it is rounded to a step of theirs; c * s
 * itself may pass them).  len_hint is the length that the work is split for (any
 * value is right).  A count or row out of range is recorded: no query is there, or
 * none sees a token.  Errors as attn_shared_prefix, and
 * UNSUPPORTED for pools that are not of the format and for more than 2^31 - 1
 * pairs of a query and a head of its group, or 2^24 - 1 workgroups (four at most
 * for each sequence, key / value head and 32 such pairs, or 1280 in all;
 * attn_cache_workspace says 0 where there are more). */
tmap_status attn_window(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, int32_t format,
                        const page_table_t* pt, const int32_t* d_rows, const int32_t* d_count, uint32_t window,
                        uint32_t sinks, uint32_t len_hint, float scale, const tmap_t* o, float* d_lse, void* d_ws,
                        uint64_t ws_bytes, void* stream);

/* Attention of drafted tokens that form a tree.  As attn_window, but the last n
 * tokens of the row are the tree's nodes: node j follows node d_parent[b * q_len
 * + j], below j, or the context itself (-1), and stands at the position of what
 * it follows and one, the context being the row's first d_lens[r] - n tokens.
 * It sees the context, the nodes on its way up and itself, each if its position
 * is within the window or below `sinks` (window 0: always).  q_len is at most
 * 1024.  A parent out of range is recorded, and its node taken to follow the
 * context; a row shorter than its tree is recorded, and its nodes see nothing.
 * Errors as attn_window. */
tmap_status attn_tree(const tmap_t* q, const tmap_t* k_pool, const tmap_t* v_pool, int32_t format,
                      const page_table_t* pt, const int32_t* d_rows, const int32_t* d_count, const int32_t* d_parent,
                      uint32_t window, uint32_t sinks, uint32_t len_hint, float scale, const tmap_t* o, float* d_lse,
                      void* d_ws, uint64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* ATT_KVCACHE_H */
