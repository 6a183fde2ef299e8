"""The paged e4m3 cache and the attention that reads it: Python entry of
include/litetopk_attend.h (same names as the C ABI, minus the prefix).

A cache is the tuple (k, v, k_scale, v_scale): k and v [n_pages, Hkv, page, D]
float8_e4m3fn, the scales [n_pages, Hkv] float32.  A batch is page_table
[B, max_pages], cu [B + 1] and kv_len [B], all int32: sequence b owns the rows
cu[b] .. cu[b+1]-1 of the call, at the last positions of its kv_len[b] tokens.

Tensors are contiguous and on the cache's device; calls run on that device's
current stream.  Wrong types raise TypeError, wrong shapes or places
ValueError, and what the library refuses LtkError.  The operators compute no
gradients: a tensor that requires grad (while grad mode is on) or carries a
tangent raises RuntimeError.
"""
from __future__ import annotations

import importlib.util
import os

from ._binding import _c_i32, _c_i64, _c_sz, LtkError, library
from .build import bind_path

ATTEND, ATTEND_SELECTED, ATTEND_PACKED = 0, 1, 2

_BIND = None


def _bind():
    """The compiled argument reader (csrc/attend_bind.cpp); raises if it has not been built."""
    global _BIND
    if _BIND is None:
        library()
        path = bind_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m indexer_topk_long_amd.build`")
        spec = importlib.util.spec_from_file_location("ltk_bind", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        _BIND = mod
    return _BIND


def kv_append(k, v, cache, page_table, cu, kv_len, inv_freq=None, q=None, interleaved: bool = False, q_out=None):
    """Appends rows to the cache in place (litetopk_kv_append).

    k and v [T, Hkv, D] bfloat16; inv_freq [rot/2] float64 (radians per
    position; None: no rotation) rotates the first rot dimensions of the keys,
    pairs (i, i + rot/2), or (2i, 2i + 1) when `interleaved`, and of the
    queries q [T, Hq, D] bfloat16 where given.  Returns the rotated queries
    (q_out, which may be q; rows outside every sequence are not written) or
    None."""
    return (_BIND or _bind()).kv_append(k, v, cache, page_table, cu, kv_len, inv_freq, q, interleaved, q_out)


def attend(q, cache, page_table, cu, kv_len, scale=None, window: int = 0, n_sink: int = 0, out=None, workspace=None):
    """Causal attention over the cache (litetopk_attend): q [T, Hq, D]
    bfloat16 -> out [T, Hq, D] bfloat16.  With window > 0 the row at position p
    sees the keys s <= p with s > p - window or s < n_sink.  scale defaults to
    1 / sqrt(D).  Rows outside every sequence are not written."""
    return (_BIND or _bind()).attend(q, cache, page_table, cu, kv_len, scale, window, n_sink, out, workspace)


def attend_selected(q, cache, page_table, cu, kv_len, idx, scale=None, out=None, workspace=None):
    """Attention of each row over its own keys idx [T, topk] int32, positions
    in its sequence as score_select returns them (litetopk_attend_selected);
    entries outside the row's causal range are no keys."""
    return (_BIND or _bind()).attend_selected(q, cache, page_table, cu, kv_len, idx, scale, out, workspace)


def attend_packed(q, cache, page_table, kv_len, shared, masks, lens, group: int, scale=None, out=None,
                  workspace=None):
    """Joint attention of groups of `group` consecutive rows over the shared
    lists of dsa_pack (litetopk_attend_packed).  One sequence: page_table
    [1, max_pages], kv_len [1], and the T rows of q are its last T tokens."""
    return (_BIND or _bind()).attend_packed(q, cache, page_table, kv_len, shared, masks, lens, group, scale, out,
                                            workspace)


def attend_workspace_bytes(kind: int, T: int, Hq: int, n_kv_heads: int, head_dim: int, n_seq: int,
                           entries: int, group: int = 0) -> int:
    """Workspace bytes that suffice for an attend call and for all with no more
    rows, sequences and entries (litetopk_attend_workspace_bytes)."""
    f = library().litetopk_attend_workspace_bytes
    f.restype, f.argtypes = _c_sz, [_c_i32] * 6 + [_c_i64, _c_i32]
    n = f(kind, T, Hq, n_kv_heads, head_dim, n_seq, entries, group)
    if n == 0:
        raise LtkError(-1, "litetopk_attend_workspace_bytes")
    return int(n)
