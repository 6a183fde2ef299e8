/*
 * litetopk_prompt.h -- C ABI of what prompts need beside the 8-bit paged cache
 * of litetopk_attend.h:
 *
 *   litetopk_attend_prompt           causal attention over whole prompts in 16
 *                                    bits, packed sequences of any lengths
 *   litetopk_attend_prompt_backward  its gradient
 *   litetopk_attend_shared           attention over the cache for sequences that
 *                                    share their first tokens, read once for all
 *   litetopk_kv_read                 rows of the cache back in 16 or 32 bits
 *
 * Conventions: those of litetopk_attend.h (device pointers, caller-owned
 * memory, asynchronous on `stream`, errors before anything is enqueued; cu and
 * lengths are read on the device, so their contents are data, never errors;
 * results do not depend on timing).
 */
#ifndef LITETOPK_PROMPT_H
#define LITETOPK_PROMPT_H

#include "litetopk_attend.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { LTK_ROWS_BF16 = 0, LTK_ROWS_FP16 = 1, LTK_ROWS_FP32 = 2 } ltk_row_type;

/* A tensor [rows, heads, head_dim] of 16-bit values: element (t, h, d) lies at
 * t * row_stride + h * head_stride + d.  Strides are multiples of 8 elements
 * (a broadcast input has 0), row strides up to 2^23 and head strides up to 2^27;
 * the address is one of 16 bytes. */
typedef struct {
    void* data;
    int64_t row_stride, head_stride;
} ltk_rows;

/* Packed prompts (HOST struct of DEVICE pointers).  Sequence b owns the rows
 * cu[b] .. cu[b+1]-1 and the keys cu_k[b] .. cu_k[b+1]-1 (both non-decreasing;
 * cu_k NULL: the same as cu, then S == T).  Its n rows sit at the last positions
 * of its m keys: row i is at position m - n + i, and sees the keys s <= its
 * position, with window > 0 only those with s > position - window.  A row that
 * sees no key (n > m), and one outside every sequence, gets zeros, the log-sum
 * -infinity, and gradients of zero.
 *
 * The q, k, v, dout of a sequence must be finite; what lies outside every
 * sequence may be anything.
 *
 *   type       LTK_ROWS_BF16 or LTK_ROWS_FP16: that of q, k, v, out and all gradients
 *   n_q_heads  a multiple of n_kv_heads; query head h reads key/value head
 *              h / (n_q_heads / n_kv_heads); fewer than 2^15 to one
 *   head_dim   64 or 128 (LTK_EUNSUPPORTED otherwise)
 *   T, S       rows of q, keys of k: T * n_q_heads and S * n_kv_heads <= 2^31 - 256
 *              (calls that would launch 2^32 threads are refused: 2 for every row and
 *              query head or key, and 256 for every sequence and key/value head)
 *   scale      finite, also times log2(e)
 *   window     >= 0 (0: none) */
typedef struct {
    const int32_t* cu;     /* [n_seq + 1] */
    const int32_t* cu_k;   /* [n_seq + 1] or NULL */
    int32_t n_seq, T, S;
    int32_t n_q_heads, n_kv_heads, head_dim, type;
    float scale;
    int32_t window;
} ltk_prompt;

/* Workspace that suffices for the call (at least 256; 0 for invalid sizes).
 * backward: 0 forward, 1 backward. */
size_t litetopk_attend_prompt_workspace_bytes(const ltk_prompt* p, int32_t backward);

/* out [T, n_q_heads, head_dim] and lse [T, n_q_heads] fp32 (the natural logarithm
 * of the sum of exp(scale q.k); may be NULL) are contiguous.  rest, like out, or
 * NULL: what the rounding of out left out, rounded itself; the backward pass
 * takes out + rest, so that the rounding of out is not in its gradients.
 *
 * Scores, statistics and sums are fp32; a weight is rounded once to the type of
 * q for its product with the value (in fp16, weights below 2^-32 of the row's
 * largest may vanish). */
int litetopk_attend_prompt(const ltk_prompt* p, const ltk_rows* q, const ltk_rows* k, const ltk_rows* v, void* out,
                           void* rest, float* lse, void* ws, size_t ws_bytes, void* stream);

/* dq [T, n_q_heads, head_dim], dk and dv [S, n_kv_heads, head_dim], contiguous,
 * from dout and what the forward call returned (rest may be NULL).  dq, or dk and
 * dv, may be NULL where they are not wanted.
 *
 * With P = exp(scale q.k - lse) and delta = dout . (out + rest):
 *   dv = P^T dout,  dS = P (dout v^T - delta),  dq = scale dS k,  dk = scale dS^T q.
 * P and dS are rounded once to the type of q for these products; sums are fp32, in
 * a fixed order.  In fp16, values of dS below 2^-25 vanish and those past 65504 are
 * infinite (scale the loss), and P is held 2^14 times its size, so that only
 * weights below 2^-39 vanish from dv. */
int litetopk_attend_prompt_backward(const ltk_prompt* p, const ltk_rows* q, const ltk_rows* k, const ltk_rows* v,
                                    const void* out, const void* rest, const float* lse, const ltk_rows* dout,
                                    void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);

/* Causal attention over the cache (no window) for sequences that share their
 * first tokens, as answers to one prompt do: the result of litetopk_attend, but
 * the shared keys are read once for all rows of a group.
 *
 *  groups      [n_group + 1] int32, non-decreasing, n_group <= 2^30: group j is the
 *              sequences groups[j] .. groups[j+1]-1; sequences in no group share
 *              nothing
 *  shared_len  [n_group] int32: tokens that the group's sequences share (clamped
 *              to the table).  Their keys are read through the page table of the
 *              group's first sequence; those from shared_len on, which may lie
 *              inside a page, through each sequence's own.  Every row of the group
 *              sees all shared keys: they lie before the rows, shared_len <=
 *              kv_len - rows for each of its sequences.  (A page that sequences
 *              have copied and appended to may have another scale in each, so for
 *              litetopk_attend's very bytes share whole pages.)
 *
 * The rest as for litetopk_attend.  Sums over the shared keys pass through the
 * workspace in fp32. */
int litetopk_attend_shared(const ltk_kv_cache* cache, const ltk_kv_batch* batch, const void* q, int32_t T, int32_t Hq,
                           const int32_t* groups, const int32_t* shared_len, int32_t n_group, float scale, void* out,
                           void* ws, size_t ws_bytes, void* stream);

/* Workspace that suffices for that call and for all of no more rows, sequences,
 * groups and entries (max_pages * page_size); 0 for invalid sizes. */
size_t litetopk_attend_shared_workspace_bytes(int32_t T, int32_t Hq, int32_t n_kv_heads, int32_t head_dim, int32_t n_seq,
                                              int32_t n_group, int64_t entries);

/* Reads rows of the cache back: k_out and v_out [T, n_kv_heads, head_dim] of
 * `type`, contiguous, 16-byte aligned, without memory in common.  Row cu[b] + i
 * holds the token at position kv_len[b] - (cu[b+1] - cu[b]) + i of sequence b, as
 * kv_append would place it: its bytes' values times the page's scale, formed in fp32
 * and rounded to `type` (exact in fp32, and in bf16 for the powers of two that
 * kv_append writes).  T may end inside a sequence: its first rows are read then.  A
 * row before its sequence's first token, past the table or on a page that is none is
 * zeros; rows outside every sequence are not written.  T * n_kv_heads <= 2^31 - 256; calls that would launch
 * 2^32 threads are refused (LTK_EINVAL): head_dim / 8 for every row. */
int litetopk_kv_read(const ltk_kv_cache* cache, const ltk_kv_batch* batch, int32_t T, int32_t type, void* k_out,
                     void* v_out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LITETOPK_PROMPT_H */
