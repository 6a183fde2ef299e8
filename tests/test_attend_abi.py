"""The C ABI of the paged cache's operators without a GPU: exports, struct
layouts, and every argument error before any device call."""
import ctypes
import os
import re
import subprocess

import pytest

import indexer_topk_long_amd as ltk
from indexer_topk_long_amd import attention as A
from indexer_topk_long_amd import build as B

_p, _i, _f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -3


class CCache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("n_pages", _i), ("n_kv_heads", _i),
                ("page_size", _i), ("head_dim", _i)]


class CBatch(ctypes.Structure):
    _fields_ = [("page_table", _p), ("cu", _p), ("kv_len", _p), ("n_seq", _i), ("max_pages", _i)]


def _fn(name):
    f = getattr(ltk.library(), name)
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(CCache), ctypes.POINTER(CBatch)] + {
        "litetopk_kv_append": [_p, _p, _p, _i, _i, _p, _i, _i, _p, _p],
        "litetopk_attend": [_p, _i, _i, _f, _i, _i, _p, _p, ctypes.c_size_t, _p],
        "litetopk_attend_selected": [_p, _i, _i, _p, _i, _f, _p, _p, ctypes.c_size_t, _p],
        "litetopk_attend_packed": [_p, _i, _i, _p, _p, _p, _i, _i, _f, _p, _p, ctypes.c_size_t, _p]}[name]
    return f


P, MIS = 0x10000, 0x10004          # aligned and misaligned fake device addresses, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.lib_path()):
        B.build()
    return ltk.library()


def test_header_functions_are_exported(lib):
    src = open(os.path.join(B.INCLUDE, "litetopk_attend.h")).read()
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(litetopk_\w+)\s*\(", src, flags=re.M)))
    assert names == ["litetopk_attend", "litetopk_attend_packed", "litetopk_attend_selected",
                     "litetopk_attend_workspace_bytes", "litetopk_kv_append"]
    for n in names:
        assert hasattr(lib, n), n


def test_header_is_c_and_matches_binding_layout(tmp_path):
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "litetopk_attend.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu\\n", sizeof(ltk_kv_cache), offsetof(ltk_kv_cache, n_pages),'
                   ' sizeof(ltk_kv_batch), offsetof(ltk_kv_batch, n_seq)); return 0;}\n')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", B.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(CCache), CCache.n_pages.offset, ctypes.sizeof(CBatch),
                   CBatch.n_seq.offset]


def _cb(kw):
    c = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=100, n_kv_heads=4, page_size=64, head_dim=128)
    b = dict(page_table=P, cu=P, kv_len=P, n_seq=3, max_pages=50)
    for d in (c, b):
        d.update({x: kw.pop(x) for x in list(kw) if x in d})
    return CCache(*c.values()), CBatch(*b.values())


CACHE_ERRORS = [
    (dict(n_pages=0), EINVAL), (dict(n_kv_heads=0), EINVAL), (dict(n_seq=-1), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(head_dim=96), EUNSUP), (dict(head_dim=256), EUNSUP), (dict(page_size=8), EUNSUP),
    (dict(page_size=48), EUNSUP), (dict(page_size=256), EUNSUP),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k_scale=None), EINVAL), (dict(v_scale=None), EINVAL),
    (dict(k=MIS), EINVAL), (dict(v=MIS), EINVAL),
    (dict(page_table=None), EINVAL), (dict(kv_len=None), EINVAL),
    (dict(n_pages=1 << 24, n_kv_heads=2), EINVAL),           # 2^31 cache rows
    (dict(max_pages=1 << 25), EINVAL),                       # 2^31 positions
    (dict(T=-1), EINVAL), (dict(T=0), OK), (dict(n_seq=0, page_table=None, kv_len=None, cu=None), OK),
]


def _append(**kw):
    c, b = _cb(kw)
    a = dict(kp=P, vp=P, q=P, T=4, Hq=8, f=P, rot=64, il=0, qo=P)
    a.update(kw)
    return _fn("litetopk_kv_append")(ctypes.byref(c), ctypes.byref(b), a["kp"], a["vp"], a["q"], a["T"], a["Hq"],
                                       a["f"], a["rot"], a["il"], a["qo"], None)


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(cu=None), EINVAL), (dict(kp=None), EINVAL), (dict(vp=None), EINVAL), (dict(kp=MIS), EINVAL),
    (dict(q=MIS), EINVAL), (dict(qo=MIS), EINVAL), (dict(qo=None), EINVAL), (dict(q=None), EINVAL),
    (dict(rot=-2), EINVAL), (dict(rot=130), EINVAL), (dict(rot=63), EINVAL), (dict(f=None), EINVAL),
    (dict(f=MIS), EINVAL), (dict(Hq=6), EINVAL), (dict(Hq=0), EINVAL),
    (dict(T=1 << 29, Hq=8), EINVAL),
    (dict(T=0, kp=None, vp=None, q=None, qo=None, f=None, rot=0), OK),
])
def test_append_argument_errors(kw, code):
    assert _append(**dict(kw)) == code


def _attend(kind, **kw):
    c, b = _cb(kw)
    a = dict(q=P, T=4, Hq=8, scale=0.1, window=0, sink=0, idx=P, topk=16, shared=P, masks=P, lens=P, group=8, cap=64,
             out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    head = (ctypes.byref(c), ctypes.byref(b), a["q"], a["T"], a["Hq"])
    tail = (a["out"], a["ws"], a["wsb"], None)
    if kind == "attend":
        return _fn("litetopk_attend")(*head, a["scale"], a["window"], a["sink"], *tail)
    if kind == "selected":
        return _fn("litetopk_attend_selected")(*head, a["idx"], a["topk"], a["scale"], *tail)
    return _fn("litetopk_attend_packed")(*head, a["shared"], a["masks"], a["lens"], a["group"], a["cap"], a["scale"],
                                           *tail)


COMMON = [(dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL), (dict(q=MIS), EINVAL),
          (dict(out=MIS), EINVAL), (dict(ws=MIS), EINVAL), (dict(scale=float("nan")), EINVAL),
          (dict(scale=float("inf")), EINVAL), (dict(Hq=6), EINVAL), (dict(Hq=0), EINVAL), (dict(wsb=255), EWS),
          (dict(T=1 << 29), EINVAL)]


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + COMMON + [
    (dict(cu=None), EINVAL), (dict(window=-1), EINVAL), (dict(sink=-1), EINVAL), (dict(T=0, q=None, out=None, ws=None), OK)])
def test_attend_argument_errors(kw, code):
    assert _attend("attend", **dict(kw)) == code


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + COMMON + [
    (dict(cu=None), EINVAL), (dict(idx=None), EINVAL), (dict(topk=0), EINVAL), (dict(topk=65537), EINVAL)])
def test_selected_argument_errors(kw, code):
    assert _attend("selected", **dict(kw)) == code


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in CACHE_ERRORS if "n_seq" not in k] + COMMON + [
    (dict(n_seq=3), EINVAL), (dict(n_seq=0), EINVAL), (dict(shared=None), EINVAL), (dict(masks=None), EINVAL),
    (dict(lens=None), EINVAL), (dict(group=0), EINVAL), (dict(group=33), EINVAL), (dict(cap=0), EINVAL),
    (dict(cap=(1 << 26) + 1), EINVAL), (dict(T=0, cu=None), OK)])
def test_packed_argument_errors(kw, code):
    assert _attend("packed", **{"n_seq": 1, **kw}) == code


def test_null_structs_are_refused():
    f = _fn("litetopk_attend")
    c, b = _cb({})
    assert f(None, ctypes.byref(b), P, 4, 8, 0.1, 0, 0, P, P, 1 << 30, None) == EINVAL
    assert f(ctypes.byref(c), None, P, 4, 8, 0.1, 0, 0, P, P, 1 << 30, None) == EINVAL


def test_workspace_sizes():
    ws = A.attend_workspace_bytes
    one = ws(A.ATTEND, 1, 64, 8, 128, 1, 1 << 20)
    assert one >= 8 * 16 * 128 * 4           # partial rows of a split call
    assert ws(A.ATTEND, 8192, 64, 8, 128, 1, 1 << 17) >= 256
    for bad in [(3, 1, 8, 8, 128, 1, 10), (0, -1, 8, 8, 128, 1, 10), (0, 1, 8, 3, 128, 1, 10),
                (0, 1, 8, 8, 96, 1, 10), (0, 1, 8, 8, 128, 1, 0), (0, 1, 8, 8, 128, -1, 10), (0, 1, 0, 8, 128, 1, 10),
                (2, 1, 8, 8, 128, 1, 10), (2, 1, 8, 8, 128, 1, 10, 33)]:
        with pytest.raises(ltk.LtkError):
            ws(*bad)


def test_a_short_workspace_is_refused():
    need = A.attend_workspace_bytes(A.ATTEND, 4, 8, 4, 128, 3, 50 * 64)
    assert _attend("attend", wsb=need - 1) == EWS
    need = A.attend_workspace_bytes(A.ATTEND_SELECTED, 4, 8, 4, 128, 3, 4096)
    assert need > 256 and _attend("selected", topk=4096, wsb=need - 1) == EWS
    need = A.attend_workspace_bytes(A.ATTEND_PACKED, 4, 8, 4, 128, 1, 4096, 8)
    assert _attend("packed", n_seq=1, cap=4096, wsb=need - 1) == EWS


def test_binding_refuses_what_the_kernels_could_not_read():
    """Shapes, types and places of tensors, checked before the library is called (CPU tensors are refused last)."""
    import torch
    f8, bf, i32 = torch.float8_e4m3fn, torch.bfloat16, torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=f8)
    s = torch.ones(4, 2)
    cache, table, cu, n = (k, k, s, s), torch.zeros(1, 4, dtype=i32), torch.tensor([0, 1], dtype=i32), torch.ones(1, dtype=i32)
    q = torch.zeros(1, 4, 64, dtype=bf)
    with pytest.raises(ValueError, match="device tensor"):
        ltk.attend(q, cache, table, cu, n)
    with pytest.raises(ValueError, match="cache must be"):
        ltk.attend(q, (k, k, s), table, cu, n)
    with pytest.raises(TypeError, match="float8"):
        ltk.attend(q, (k.float(), k, s, s), table, cu, n)
    with pytest.raises(ValueError, match=r"cache k must be"):
        ltk.attend(q, (k[0], k, s, s), table, cu, n)


@pytest.mark.parametrize("kind", ["attend", "selected", "packed"])
def test_a_score_scale_that_overflows_in_base_2_is_refused(kind):
    assert _attend(kind, scale=3.0e38) == EINVAL


def test_a_group_of_more_pairs_than_are_numbered_is_refused():
    assert _attend("packed", n_seq=1, T=1, Hq=1 << 28, group=32) == EINVAL
    with pytest.raises(ltk.LtkError):
        ltk.attend_workspace_bytes(2, 1, 1 << 28, 4, 128, 1, 64, 32)
