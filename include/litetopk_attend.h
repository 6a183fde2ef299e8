/*
 * litetopk_attend.h -- C ABI of the 8-bit paged key/value cache and the
 * attention that reads it: what a decode step or a prefill chunk runs around
 * the key selection of litetopk.h.
 *
 *   litetopk_kv_append        rotates new keys by their positions, quantises
 *                             keys and values and writes them to the cache
 *   litetopk_attend           causal attention over a sequence, optionally
 *                             with a sliding window and visible first tokens
 *   litetopk_attend_selected  each row over its own key list (the result of
 *                             litetopk_score_select)
 *   litetopk_attend_packed    groups of rows over shared lists with row masks
 *                             (the result of litetopk_dsa_pack)
 *
 * Attention of the row at position p over the keys s it sees, per query head:
 *   x_s = scale * (q . k_s)     out = sum_s exp(x_s) v_s / sum_s exp(x_s)
 * A row that sees no key gets zeros.  Query head h reads key/value head
 * h / (Hq / n_kv_heads).  T * Hq <= 2^31 - 256.
 *
 * Conventions: those of litetopk.h (device pointers, caller-owned memory,
 * asynchronous on `stream`, errors before anything is enqueued).  q, k, v and
 * out are bf16, 16-byte aligned.  cu, kv_len, page_table and key lists are
 * read on the device, so their contents are data, never errors:
 *  - a page id outside [0, n_pages) or a position past the table is no page:
 *    rows are not written there and its keys are not seen;
 *  - rows outside every sequence (at or past cu[n_seq]) are not written;
 *  - a list entry outside [0, kv_len) or after the row's position is no key.
 * Calls that would launch 2^32 threads are refused (LTK_EINVAL): selected and
 * packed ones launch 256 for 16 or more (row, head) pairs of a list and key/value
 * head.
 *
 * Bytes and scales that hold no key of the sequence may be anything (NaN
 * included); everything else must be finite, scales also within 2^-64 .. 2^64,
 * the range that the append writes (the ends of it may meet in one sequence).
 *
 * Sums, softmax statistics and partial rows are fp32, products of bf16 and
 * fp16 operands (the cache's bytes convert exactly).  A key's weight times its
 * value scale is rounded to fp16 relative to the row's largest such product:
 * 2^-11 of itself, or 2^-25 of the largest where it is below fp16's normal
 * range (2^-14 of it).  With many rows a key, some are rounded twice (a larger
 * product met in the same 64 keys): 2^-10, or 2^-24 of the largest.  Results do
 * not depend on timing: the same call gives the same bits.
 */
#ifndef LITETOPK_ATTEND_H
#define LITETOPK_ATTEND_H

#include "litetopk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Paged cache (HOST struct of DEVICE pointers).  A page holds page_size
 * consecutive tokens of one sequence:
 *   k, v              [n_pages, n_kv_heads, page_size, head_dim] e4m3fn
 *   k_scale, v_scale  [n_pages, n_kv_heads] fp32; a byte stands for its e4m3
 *                     value times its page's and head's scale
 * page_size in {16, 32, 64, 128}, head_dim in {64, 128} (LTK_EUNSUPPORTED
 * otherwise), n_pages * n_kv_heads * page_size < 2^31; 16-byte aligned. */
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int32_t n_pages, n_kv_heads, page_size, head_dim;
} ltk_kv_cache;

/* Batch of sequences (HOST struct of DEVICE pointers).  Sequence b owns the
 * rows cu[b] .. cu[b+1]-1 of the call (cu non-decreasing), which sit at its
 * last positions: row cu[b] + i is at position kv_len[b] - (cu[b+1] - cu[b]) + i.
 * kv_len counts the rows of the call.  Token s of sequence b is in page
 * page_table[b][s / page_size], slot s % page_size.
 * n_seq >= 0, max_pages >= 1, max_pages * page_size <= 2^31 - 128 (key offsets
 * past a tile's end stay in int32). */
typedef struct {
    const int32_t* page_table;   /* [n_seq, max_pages] */
    const int32_t* cu;           /* [n_seq + 1] */
    const int32_t* kv_len;       /* [n_seq] */
    int32_t n_seq, max_pages;
} ltk_kv_batch;

typedef enum {
    LTK_ATTEND = 0,
    LTK_ATTEND_SELECTED = 1,
    LTK_ATTEND_PACKED = 2
} ltk_attend_kind;

/* Appends the rows' keys and values to the cache.
 *
 *  k, v      [T, n_kv_heads, head_dim] bf16
 *  q, q_out  [T, Hq, head_dim] bf16: queries to rotate, or both NULL (Hq
 *            ignored); q_out may be q
 *  inv_freq  [rot_dim / 2] fp64 rotation frequencies in radians per position,
 *            or NULL with rot_dim == 0 (no rotation)
 *  rot_dim   even, 0 .. head_dim: the first rot_dim dimensions are rotated,
 *            dimension pair (i, i + rot_dim/2), or (2i, 2i + 1) when
 *            `interleaved`, by position * inv_freq[i]
 *
 * Angles are formed in fp64.  Rotated keys are rounded once to fp32 and once
 * to e4m3, queries once to bf16.
 *
 * A page's scale is the least power of two s (2^-64 .. 2^64) with
 * |x| <= 448 s for every token of the page.  When the rows join a page that
 * already holds tokens of the sequence, its scale never falls; if it grows,
 * the bytes of the tokens before the rows are rounded again to the new scale
 * (exact for a power of two, except for e4m3 subnormals).  A page begun with a
 * scale that is no power of two keeps it until it grows.  A page written from its first slot
 * starts a new scale.  Slots behind the last row are left as they are.
 * No page may receive rows twice in one call: from two sequences, or at two places
 * of a sequence's table. */
int litetopk_kv_append(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* k, const void* v,
                       const void* q, int32_t T, int32_t Hq, const double* inv_freq, int32_t rot_dim,
                       int32_t interleaved, void* q_out, void* stream);

/* Bytes of workspace that suffice for an attend call of `kind` and for every call
 * of it with no more rows, sequences and entries and the same heads and group (at
 * least 256; 0 for invalid sizes).  Smaller calls may need more than larger ones:
 * their work is cut into more parts.  `entries` bounds the keys a row reads: max_pages *
 * page_size (attend), topk (selected) or cap (packed); `group` is the packed
 * call's (ignored otherwise). */
size_t litetopk_attend_workspace_bytes(int32_t kind, int32_t T, int32_t Hq, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t n_seq, int64_t entries, int32_t group);

/* Causal attention: the row at position p sees the keys s <= p, and with
 * window > 0 only those with s > p - window or s < n_sink.
 *
 *  q, out  [T, Hq, head_dim] bf16, Hq a multiple of n_kv_heads
 *  scale   finite, also times log2(e)
 *  window  >= 0 (0: no window); n_sink >= 0 (no effect without a window) */
int litetopk_attend(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T, int32_t Hq,
                    float scale, int32_t window, int32_t n_sink, void* out, void* ws, size_t ws_bytes, void* stream);

/* Attention of each row over its own list idx [T, topk] int32 of positions in
 * its sequence, in any order (1 <= topk <= 65536).  Entries are distinct; one
 * that repeats counts each time. */
int litetopk_attend_selected(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T,
                             int32_t Hq, const int32_t* idx, int32_t topk, float scale, void* out, void* ws,
                             size_t ws_bytes, void* stream);

/* Joint attention of groups of consecutive rows of ONE sequence (n_seq == 1;
 * cu is ignored: the T rows are the sequence's last T tokens).  Row t belongs
 * to group g = t / group and sees shared[g][j], j < lens[g], when bit
 * t % group of masks[g][j] is set and the key is not after it.
 *
 *  shared  [ceil(T / group), cap] int32 distinct positions per group
 *  masks   [ceil(T / group), cap] uint32; lens [ceil(T / group)] int32
 *          (clamped to [0, cap])
 *  group   1 .. 32, group * Hq / n_kv_heads <= 2^30; cap 1 .. 2^26 */
int litetopk_attend_packed(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T,
                           int32_t Hq, const int32_t* shared, const uint32_t* masks, const int32_t* lens,
                           int32_t group, int32_t cap, float scale, void* out, void* ws, size_t ws_bytes,
                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LITETOPK_ATTEND_H */
