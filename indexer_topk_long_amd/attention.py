"""ctypes binding of the paged e4m3 cache and the attention that reads it
(include/litetopk_attend.h; same names as the C ABI, minus the prefix).

A cache is the tuple (k, v, k_scale, v_scale): k and v [n_pages, Hkv, page, D]
float8_e4m3fn, the scales [n_pages, Hkv] float32.  A batch is page_table
[B, max_pages], cu [B + 1] and kv_len [B], all int32: sequence b owns the rows
cu[b] .. cu[b+1]-1 of the call, at the last positions of its kv_len[b] tokens.
"""
from __future__ import annotations

import ctypes
import functools

from ._binding import _c_i32, _c_i64, _c_p, _c_sz, LtkError, _expect, library

ATTEND, ATTEND_SELECTED, ATTEND_PACKED = 0, 1, 2


class _CCache(ctypes.Structure):
    _fields_ = [("k", _c_p), ("v", _c_p), ("k_scale", _c_p), ("v_scale", _c_p), ("n_pages", _c_i32),
                ("n_kv_heads", _c_i32), ("page_size", _c_i32), ("head_dim", _c_i32)]


class _CBatch(ctypes.Structure):
    _fields_ = [("page_table", _c_p), ("cu", _c_p), ("kv_len", _c_p), ("n_seq", _c_i32), ("max_pages", _c_i32)]


_FN = {}


def _fn(name: str):
    """A function of the library with its argument types set."""
    if name not in _FN:
        f = getattr(library(), name)
        head = [ctypes.POINTER(_CCache), ctypes.POINTER(_CBatch)]
        f.restype = ctypes.c_int
        if name == "litetopk_kv_append":
            f.argtypes = head + [_c_p, _c_p, _c_p, _c_i32, _c_i32, _c_p, _c_i32, _c_i32, _c_p, _c_p]
        elif name == "litetopk_attend":
            f.argtypes = head + [_c_p, _c_i32, _c_i32, ctypes.c_float, _c_i32, _c_i32, _c_p, _c_p, _c_sz, _c_p]
        elif name == "litetopk_attend_selected":
            f.argtypes = head + [_c_p, _c_i32, _c_i32, _c_p, _c_i32, ctypes.c_float, _c_p, _c_p, _c_sz, _c_p]
        elif name == "litetopk_attend_packed":
            f.argtypes = head + [_c_p, _c_i32, _c_i32, _c_p, _c_p, _c_p, _c_i32, _c_i32, ctypes.c_float, _c_p, _c_p,
                                 _c_sz, _c_p]
        else:
            f.restype = _c_sz
            f.argtypes = [_c_i32] * 6 + [_c_i64, _c_i32]
        _FN[name] = f
    return _FN[name]


def _refuse(t, name, dtype, shape, device):
    """Raises the first thing wrong with a tensor: type, shape (None: any size), layout, device."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if len(t.shape) != len(shape) or any(w is not None and w != n for n, w in zip(t.shape, shape)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        raise ValueError(f"{name} must be [{want}], got {tuple(t.shape)}")
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous device tensor")
    raise ValueError(f"{name} is on {t.device}, the cache on cuda:{device}: all tensors must share one device")


def _check(t, name, dtype, shape, device):
    """The address of a contiguous tensor of exactly this dtype, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, shape, device)


def _cache(cache):
    """(ltk_kv_cache, device index) of a (k, v, k_scale, v_scale)."""
    import torch
    _expect(isinstance(cache, (tuple, list)) and len(cache) == 4, "cache must be (k, v, k_scale, v_scale)")
    k, v, ks, vs = cache
    f8, f32, shape, dev = torch.float8_e4m3fn, torch.float32, k.shape, k.get_device()
    if k.dtype is not f8 or len(shape) != 4 or dev < 0 or not k.is_contiguous():
        _refuse(k, "cache k", f8, (None,) * 4, dev)
    n, hkv, page, d = shape
    per = (n, hkv)
    return _CCache(k.data_ptr(), _check(v, "cache v", f8, shape, dev), _check(ks, "k_scale", f32, per, dev),
                   _check(vs, "v_scale", f32, per, dev), n, hkv, page, d), dev


def _batch(page_table, cu, kv_len, dev):
    import torch
    i32 = torch.int32
    if len(page_table.shape) != 2:
        _refuse(page_table, "page_table", i32, (None, None), dev)
    B, mp = page_table.shape
    pt = _check(page_table, "page_table", i32, (B, mp), dev)
    pc = None if cu is None else _check(cu, "cu", i32, (B + 1,), dev)
    return _CBatch(pt, pc, _check(kv_len, "kv_len", i32, (B,), dev), B, mp)


class _On:
    """The library launches on the current device: makes `device` current for a
    call where it is not, and names its current stream."""

    def __init__(self, device):
        import torch
        self.torch, self.index, self.was = torch, device, torch.cuda.current_device()

    def __enter__(self):
        if self.was != self.index:
            self.torch.cuda.set_device(self.index)
        return self.torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.was != self.index:
            self.torch.cuda.set_device(self.was)


def _raise(rc, where):
    if rc != 0:
        raise LtkError(rc, where)


def kv_append(k, v, cache, page_table, cu, kv_len, inv_freq=None, q=None, interleaved: bool = False, q_out=None):
    """Appends rows to the cache in place (litetopk_kv_append).

    k and v [T, Hkv, D] bfloat16; inv_freq [rot/2] float64 (radians per
    position; None: no rotation) rotates the first rot dimensions of the keys,
    pairs (i, i + rot/2), or (2i, 2i + 1) when `interleaved`, and of the
    queries q [T, Hq, D] bfloat16 where given.  Returns the rotated queries
    (q_out, which may be q; rows outside every sequence are not written) or
    None."""
    import torch
    c, dev = _cache(cache)
    b = _batch(page_table, cu, kv_len, dev)
    T, bf16 = k.shape[0], torch.bfloat16
    rows = (T, c.n_kv_heads, c.head_dim)
    pk, pv = _check(k, "k", bf16, rows, dev), _check(v, "v", bf16, rows, dev)
    pf, rot = None, 0
    if inv_freq is not None:
        half = inv_freq.numel()
        pf, rot = _check(inv_freq, "inv_freq", torch.float64, (half,), dev), 2 * half
    pq = po = None
    Hq = 0
    if q is not None:
        Hq = q.shape[1] if len(q.shape) == 3 else None
        pq = _check(q, "q", bf16, (T, Hq, c.head_dim), dev)
        if q_out is None:
            q_out = torch.empty_like(q)
        po = _check(q_out, "q_out", bf16, q.shape, dev)
    else:
        _expect(q_out is None, "q_out without q")
    with _On(dev) as stream:
        _raise(_fn("litetopk_kv_append")(ctypes.byref(c), ctypes.byref(b), pk, pv, pq, T, Hq, pf, rot,
                                         int(bool(interleaved)), po, stream), "litetopk_kv_append")
    return q_out


@functools.lru_cache(maxsize=1024)   # sizes only
def attend_workspace_bytes(kind: int, T: int, Hq: int, n_kv_heads: int, head_dim: int, n_seq: int,
                           entries: int, group: int = 0) -> int:
    """Workspace bytes of an attend call (litetopk_attend_workspace_bytes)."""
    n = _fn("litetopk_attend_workspace_bytes")(kind, T, Hq, n_kv_heads, head_dim, n_seq, entries, group)
    if n == 0:
        raise LtkError(-1, "litetopk_attend_workspace_bytes")
    return int(n)


def _queries(q, c, scale, out, dev):
    import torch
    T, Hq = q.shape[:2] if len(q.shape) == 3 else (None, 0)
    pq = _check(q, "q", torch.bfloat16, (T, Hq, c.head_dim), dev)
    _expect(Hq >= 1 and Hq % max(c.n_kv_heads, 1) == 0, f"q has {Hq} heads, the cache {c.n_kv_heads}: not a multiple")
    if out is None:
        out = torch.empty_like(q)
        po = out.data_ptr()
    else:
        po = _check(out, "out", torch.bfloat16, q.shape, dev)
    return pq, T, Hq, po, out, (c.head_dim ** -0.5 if scale is None else float(scale))


def _space(kind, T, Hq, c, n_seq, entries, workspace, dev, group=0):
    """(address, bytes, tensor) of the call's workspace."""
    need = attend_workspace_bytes(kind, T, Hq, c.n_kv_heads, c.head_dim, n_seq, entries, group)
    if workspace is None:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
        return workspace.data_ptr(), need, workspace
    size = workspace.numel() * workspace.element_size()
    if size < need:
        raise ValueError(f"workspace too small: {size} bytes, {need} needed")
    return _check(workspace, "workspace", workspace.dtype, workspace.shape, dev), size, workspace


def attend(q, cache, page_table, cu, kv_len, scale=None, window: int = 0, n_sink: int = 0, out=None, workspace=None):
    """Causal attention over the cache (litetopk_attend): q [T, Hq, D]
    bfloat16 -> out [T, Hq, D] bfloat16.  With window > 0 the row at position p
    sees the keys s <= p with s > p - window or s < n_sink.  scale defaults to
    1 / sqrt(D).  Rows outside every sequence are not written."""
    c, dev = _cache(cache)
    b = _batch(page_table, cu, kv_len, dev)
    pq, T, Hq, po, out, scale = _queries(q, c, scale, out, dev)
    pw, nw, workspace = _space(ATTEND, T, Hq, c, b.n_seq, max(b.max_pages * c.page_size, 1), workspace, dev)
    with _On(dev) as stream:
        _raise(_fn("litetopk_attend")(ctypes.byref(c), ctypes.byref(b), pq, T, Hq, scale, window, n_sink, po, pw, nw,
                                      stream), "litetopk_attend")
    return out


def attend_selected(q, cache, page_table, cu, kv_len, idx, scale=None, out=None, workspace=None):
    """Attention of each row over its own keys idx [T, topk] int32, positions
    in its sequence as score_select returns them (litetopk_attend_selected);
    entries outside the row's causal range are no keys."""
    import torch
    c, dev = _cache(cache)
    b = _batch(page_table, cu, kv_len, dev)
    pq, T, Hq, po, out, scale = _queries(q, c, scale, out, dev)
    topk = idx.shape[1] if len(idx.shape) == 2 else None
    pi = _check(idx, "idx", torch.int32, (T, topk), dev)
    _expect(1 <= topk <= 65536, f"idx must hold 1 to 65536 keys a row, got {topk}")
    pw, nw, workspace = _space(ATTEND_SELECTED, T, Hq, c, b.n_seq, topk, workspace, dev)
    with _On(dev) as stream:
        _raise(_fn("litetopk_attend_selected")(ctypes.byref(c), ctypes.byref(b), pq, T, Hq, pi, topk, scale, po, pw,
                                               nw, stream), "litetopk_attend_selected")
    return out


def attend_packed(q, cache, page_table, kv_len, shared, masks, lens, group: int, scale=None, out=None,
                  workspace=None):
    """Joint attention of groups of `group` consecutive rows over the shared
    lists of dsa_pack (litetopk_attend_packed).  One sequence: page_table
    [1, max_pages], kv_len [1], and the T rows of q are its last T tokens."""
    import torch
    c, dev = _cache(cache)
    b = _batch(page_table, None, kv_len, dev)
    _expect(b.n_seq == 1, f"attend_packed takes one sequence, got {b.n_seq}")
    _expect(1 <= group <= 32, f"group must lie in 1 .. 32, got {group}")
    pq, T, Hq, po, out, scale = _queries(q, c, scale, out, dev)
    ng = (T + group - 1) // group
    cap = shared.shape[1] if len(shared.shape) == 2 else None
    ps = _check(shared, "shared", torch.int32, (ng, cap), dev)
    _expect(1 <= cap <= 1 << 26, f"shared must hold 1 to 2^26 entries a group, got {cap}")
    pm = _check(masks, "masks", torch.uint32, (ng, cap), dev)
    pl = _check(lens, "lens", torch.int32, (ng,), dev)
    pw, nw, workspace = _space(ATTEND_PACKED, T, Hq, c, 1, cap, workspace, dev, group)
    with _On(dev) as stream:
        _raise(_fn("litetopk_attend_packed")(ctypes.byref(c), ctypes.byref(b), pq, T, Hq, ps, pm, pl, group, cap, scale,
                                             po, pw, nw, stream), "litetopk_attend_packed")
    return out
