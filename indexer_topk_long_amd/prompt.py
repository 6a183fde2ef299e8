"""Prompts in 16 bits beside the paged e4m3 cache: Python entry of
include/litetopk_prompt.h (same names as the C ABI, minus the prefix).

Tensors are on one device; calls run on that device's current stream.  Wrong
types raise TypeError, wrong shapes or places ValueError, and what the library
refuses LtkError.
"""
from __future__ import annotations

from . import attention as _attention


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
    raises RuntimeError.  While a stream is captured, a leaf that an eager graph on
    another stream still holds is refused too."""
    return _bind().attend_prompt(q, k, v, cu, cu_k, scale, window, return_lse)


def kv_read(cache, page_table, cu, kv_len, T: int, dtype=None, out=None):
    """Rows of the cache back (litetopk_kv_read): (k, v), each [T, Hkv, D] of
    dtype (bfloat16, the default, float16 or float32).  Row cu[b] + i is the token
    at position kv_len[b] - (cu[b+1] - cu[b]) + i of sequence b, where kv_append
    puts a row of that number; rows without a token are zeros.  out is a pair of
    tensors to write to.  Rows outside every sequence are not written."""
    if dtype is None:
        import torch
        dtype = torch.bfloat16
    return _bind().kv_read(cache, page_table, cu, kv_len, T, dtype, out)
