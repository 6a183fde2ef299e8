"""Prompts in 16 bits beside the paged e4m3 cache: Python entry of
include/litetopk_prompt.h (same names as the C ABI, minus the prefix).

Tensors are on one device; calls run on that device's current stream.  Wrong
types raise TypeError, wrong shapes or places ValueError, and what the library
refuses LtkError.
"""
from __future__ import annotations

from . import attention as _attention
from ._binding import _c_i32, _c_i64, _c_sz, LtkError, library


def _bind():
    return _attention._BIND or _attention._bind()


def attend_prompt(q, k, v, cu, cu_k=None, scale=None, window: int = 0, return_lse: bool = False):
    """Causal attention over packed prompts (litetopk_attend_prompt).

    q [T, Hq, D], k and v [S, Hkv, D], all bfloat16 or all float16, D 64 or 128,
    Hq a multiple of Hkv; views of a fused projection are taken as they lie (any
    row and head strides that are multiples of 8; others are copied).  Sequence b
    owns the rows cu[b] .. cu[b+1]-1 and the keys cu_k[b] .. cu_k[b+1]-1 (int32;
    cu_k None: the same as cu).  Its rows sit at the last positions of its keys;
    the row at position p sees the keys s <= p, with window > 0 only those with
    s > p - window.  scale defaults to 1 / sqrt(D).

    Returns out [T, Hq, D] in q's type, with return_lse also the log-sums of the
    scores [T, Hq] float32 (-inf for a row that sees nothing; no gradient flows
    through them).  Rows that see no key, and rows outside every sequence, are
    zeros.

    Differentiable in q, k and v, once: a second derivative or a forward one
    raises RuntimeError.  While a stream is captured, inputs that depend on a leaf
    which an eager graph of the default stream still holds are refused too (but under
    torch.no_grad()): the captured backward pass would end the process."""
    return _bind().attend_prompt(q, k, v, cu, cu_k, scale, window, return_lse)


def attend_shared(q, cache, page_table, cu, kv_len, groups, shared_len, scale=None, out=None, workspace=None):
    """attend for sequences that share their first tokens, as answers to one
    prompt do (litetopk_attend_shared): the same result without a window, but the
    shared keys are read once for all rows of a group.

    q, cache, page_table, cu and kv_len as for attend.  Group j is the sequences
    groups[j] .. groups[j+1]-1 (int32 [n_group + 1], non-decreasing) and shares its
    first shared_len[j] tokens (int32 [n_group]): they are read through the page
    table of its first sequence, and lie before every row of the group.  Tokens
    from shared_len[j] on, which may lie inside a page, are each sequence's own.
    Sequences in no group share nothing.  Rows outside every sequence are not
    written."""
    return _bind().attend_shared(q, cache, page_table, cu, kv_len, groups, shared_len, scale, out, workspace)


def attend_shared_workspace_bytes(T: int, Hq: int, n_kv_heads: int, head_dim: int, n_seq: int, n_group: int,
                                  entries: int) -> int:
    """Workspace bytes that suffice for an attend_shared call and for all with no
    more rows, sequences, groups and entries (litetopk_attend_shared_workspace_bytes)."""
    f = library().litetopk_attend_shared_workspace_bytes
    f.restype, f.argtypes = _c_sz, [_c_i32] * 6 + [_c_i64]
    n = f(T, Hq, n_kv_heads, head_dim, n_seq, n_group, entries)
    if n == 0:
        raise LtkError(-1, "litetopk_attend_shared_workspace_bytes")
    return int(n)


def kv_read(cache, page_table, cu, kv_len, T: int, dtype=None, out=None):
    """Rows of the cache back (litetopk_kv_read): (k, v), each [T, Hkv, D] of
    dtype (bfloat16, the default, float16 or float32).  Row cu[b] + i is the token
    at position kv_len[b] - (cu[b+1] - cu[b]) + i of sequence b, where kv_append
    puts a row of that number; T may end inside a sequence, whose first rows are read
    then.  Rows without a token are zeros.  out is a pair of tensors to write to,
    which share no memory.  Rows outside every sequence are not written."""
    if dtype is None:
        import torch
        dtype = torch.bfloat16
    return _bind().kv_read(cache, page_table, cu, kv_len, T, dtype, out)
