"""The C ABI of the prompts' operators without a GPU: exports, struct layouts, and
every argument error before any device call."""
import ctypes
import os
import re
import subprocess

import pytest

import indexer_topk_long_amd as ltk
from indexer_topk_long_amd import build as B
from tests.test_attend_abi import CACHE_ERRORS, EINVAL, EUNSUP, EWS, MIS, OK, P, CBatch, CCache, _cb

_p, _i, _f, _l, _z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_int64, ctypes.c_size_t


class CRows(ctypes.Structure):
    _fields_ = [("data", _p), ("row_stride", _l), ("head_stride", _l)]


class CPrompt(ctypes.Structure):
    _fields_ = [("cu", _p), ("cu_k", _p), ("n_seq", _i), ("T", _i), ("S", _i), ("n_q_heads", _i), ("n_kv_heads", _i),
                ("head_dim", _i), ("type", _i), ("scale", _f), ("window", _i)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.lib_path()):
        B.build()
    return ltk.library()


def test_header_functions_are_exported(lib):
    src = open(os.path.join(B.INCLUDE, "litetopk_prompt.h")).read()
    names = sorted(set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b(litetopk_\w+)\s*\(", src, flags=re.M)))
    assert names == ["litetopk_attend_prompt", "litetopk_attend_prompt_backward",
                     "litetopk_attend_prompt_workspace_bytes", "litetopk_attend_shared",
                     "litetopk_attend_shared_workspace_bytes", "litetopk_kv_read"]
    for n in names:
        assert hasattr(lib, n), n


def test_header_is_c_and_layouts(tmp_path):
    src = tmp_path / "probe.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "litetopk_prompt.h"\n'
                   'int main(void){printf("%zu %zu %zu %zu %zu\\n", sizeof(ltk_rows), sizeof(ltk_prompt),'
                   ' offsetof(ltk_prompt, n_seq), offsetof(ltk_prompt, scale), offsetof(ltk_prompt, window)); return 0;}\n')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", B.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(CRows), ctypes.sizeof(CPrompt), CPrompt.n_seq.offset, CPrompt.scale.offset,
                   CPrompt.window.offset]


def _prompt(kw):
    a = dict(cu=P, cu_k=P, n_seq=3, T=40, S=60, n_q_heads=8, n_kv_heads=2, head_dim=128, type=0, scale=0.1, window=0)
    a.update({x: kw.pop(x) for x in list(kw) if x in a})
    return CPrompt(*a.values())


def _rows(kw, name, heads):
    r = CRows(P, heads * 128, 128)
    for f in ("data", "row_stride", "head_stride"):
        if f"{name}_{f}" in kw:
            setattr(r, f, kw.pop(f"{name}_{f}"))
    return ctypes.byref(r)


def _forward(**kw):
    p = _prompt(kw)
    q, k, v = (_rows(kw, n, h) for n, h in (("q", 8), ("k", 2), ("v", 2)))
    a = dict(out=P, rest=None, lse=None, ws=P, wsb=1 << 40)
    a.update(kw)
    f = ltk.library().litetopk_attend_prompt
    f.restype, f.argtypes = ctypes.c_int, [_p] * 7 + [_p, _z, _p]
    return f(ctypes.byref(p), q, k, v, a["out"], a["rest"], a["lse"], a["ws"], a["wsb"], None)


def _backward(**kw):
    p = _prompt(kw)
    q, k, v, d = (_rows(kw, n, h) for n, h in (("q", 8), ("k", 2), ("v", 2), ("dout", 8)))
    a = dict(out=P, rest=None, lse=P, dq=P, dk=P, dv=P, ws=P, wsb=1 << 40)
    a.update(kw)
    f = ltk.library().litetopk_attend_prompt_backward
    f.restype, f.argtypes = ctypes.c_int, [_p] * 12 + [_z, _p]
    return f(ctypes.byref(p), q, k, v, a["out"], a["rest"], a["lse"], d, a["dq"], a["dk"], a["dv"], a["ws"], a["wsb"], None)


EMPTY = dict(T=0, S=0, q_data=None, k_data=None, v_data=None, out=None, ws=None, cu=None, cu_k=None, n_seq=0)
SHAPES = [
    (dict(n_seq=-1), EINVAL), (dict(T=-1), EINVAL), (dict(S=-1), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(n_q_heads=0), EINVAL), (dict(n_q_heads=7), EINVAL), (dict(head_dim=96), EUNSUP), (dict(head_dim=256), EUNSUP),
    (dict(type=2), EUNSUP), (dict(type=-1), EUNSUP), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(scale=3e38), EINVAL), (dict(window=-1), EINVAL), (dict(T=1 << 28), EINVAL), (dict(S=1 << 30), EINVAL),
    (dict(n_q_heads=1 << 15, n_kv_heads=1), EINVAL), (dict(cu_k=None), EINVAL), (dict(cu=None), EINVAL),
    (dict(q_data=None), EINVAL), (dict(k_data=None), EINVAL), (dict(v_data=None), EINVAL), (dict(q_data=MIS), EINVAL),
    (dict(k_data=MIS), EINVAL), (dict(v_data=MIS), EINVAL), (dict(q_row_stride=1028), EINVAL),
    (dict(k_head_stride=12), EINVAL), (dict(v_row_stride=-8), EINVAL), (dict(q_head_stride=-8), EINVAL),
    (dict(k_row_stride=(1 << 23) + 8), EINVAL), (dict(q_head_stride=(1 << 40) + 8), EINVAL),
    (dict(ws=None), EINVAL), (dict(ws=MIS), EINVAL), (dict(wsb=255), EWS), (dict(out=MIS), EINVAL),
    (dict(rest=MIS), EINVAL), (dict(out=None), EINVAL),
]


@pytest.mark.parametrize("kw,code", SHAPES + [(dict(lse=P + 2), EINVAL), (EMPTY, OK)])
def test_forward_argument_errors(kw, code):
    assert _forward(**dict(kw)) == code


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(lse=None), EINVAL), (dict(lse=P + 2), EINVAL), (dict(dk=None), EINVAL), (dict(dv=None), EINVAL),
    (dict(dq=MIS), EINVAL), (dict(dk=MIS), EINVAL), (dict(dv=MIS), EINVAL), (dict(dout_data=None), EINVAL),
    (dict(dout_data=MIS), EINVAL), (dict(dout_row_stride=4), EINVAL), (dict(q_head_stride=1 << 30), EINVAL),
    (dict(dout_head_stride=1 << 30), EINVAL), (dict(dq=None, dk=None, dv=None), OK),
    (dict(EMPTY, lse=None, dout_data=None, dq=None, dk=None, dv=None), OK)])
def test_backward_argument_errors(kw, code):
    assert _backward(**dict(kw)) == code


def _bytes(backward, **kw):
    f = ltk.library().litetopk_attend_prompt_workspace_bytes
    f.restype, f.argtypes = _z, [_p, _i]
    return f(ctypes.byref(_prompt(kw)), backward)


def test_workspace_bytes():
    for back in (0, 1):
        assert _bytes(back) >= 256 and _bytes(back, T=0, S=0) == 256
        for bad in (dict(T=-1), dict(n_q_heads=7), dict(head_dim=96), dict(window=-1), dict(n_seq=-1)):
            assert _bytes(back, **bad) == 0
    assert _bytes(1) >= 2 * 40 * 8 * 4                                  # two numbers for every row and head
    # the size asked for suffices for the call at both ends of the range
    for T, seqs, hq, hkv, d, w in ((1, 1, 1, 1, 64, 0), (16384, 1, 64, 8, 128, 0), (8192, 1, 32, 8, 128, 1024),
                                   ((1 << 31) - 2048, 1, 1, 1, 64, 0), (1 << 20, 1 << 20, 2, 1, 64, 0)):
        kw = dict(T=T, S=T, n_seq=seqs, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, window=w)
        need = _bytes(0, **kw), _bytes(1, **kw)
        assert all(need) and max(need) < 1 << 40
        assert _forward(**dict(kw, n_seq=1 << 24, n_kv_heads=hq)) == EINVAL          # 2^32 threads
        assert _forward(**kw, wsb=need[0] - 1) == EWS and _backward(**kw, wsb=need[1] - 1) == EWS


def _shared(**kw):
    c, b = _cb(kw)
    a = dict(q=P, T=4, Hq=8, groups=P, lens=P, n_group=2, scale=0.1, out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    f = ltk.library().litetopk_attend_shared
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(CCache), ctypes.POINTER(CBatch), _p, _i, _i, _p, _p, _i, _f, _p, _p, _z, _p]
    return f(ctypes.byref(c), ctypes.byref(b), a["q"], a["T"], a["Hq"], a["groups"], a["lens"], a["n_group"], a["scale"],
             a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(cu=None), EINVAL), (dict(groups=None), EINVAL), (dict(lens=None), EINVAL), (dict(n_group=-1), EINVAL),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL), (dict(q=MIS), EINVAL), (dict(ws=MIS), EINVAL),
    (dict(Hq=6), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(wsb=255), EWS), (dict(n_group=0, wsb=255), EWS),
    (dict(T=0, groups=None, lens=None), OK)])
def test_shared_argument_errors(kw, code):
    assert _shared(**dict(kw)) == code


def test_shared_workspace_bytes():
    f = ltk.attend_shared_workspace_bytes
    small = f(4, 8, 2, 64, 4, 1, 1024)
    assert small >= 4 * 8 * 68 * 4
    assert f(8, 8, 2, 64, 4, 1, 1024) >= small and f(4, 8, 2, 64, 4, 1, 65536) >= small
    for bad in ((-1, 8, 2, 64, 4, 1, 1024), (4, 7, 2, 64, 4, 1, 1024), (4, 8, 2, 96, 4, 1, 1024), (4, 8, 2, 64, -1, 1, 1024),
                (4, 8, 2, 64, 4, -1, 1024), (4, 8, 2, 64, 4, 1, 0)):
        with pytest.raises(ltk.LtkError):
            f(*bad)


def _read(**kw):
    c, b = _cb(kw)
    a = dict(T=4, type=0, k=P, v=P)
    kk = {x: kw.pop(x) for x in list(kw) if x in ("ko", "vo")}
    a.update(kw)
    f = ltk.library().litetopk_kv_read
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(CCache), ctypes.POINTER(CBatch), _i, _i, _p, _p, _p]
    return f(ctypes.byref(c), ctypes.byref(b), a["T"], a["type"], kk.get("ko", P), kk.get("vo", P), None)


@pytest.mark.parametrize("kw,code", CACHE_ERRORS + [
    (dict(cu=None), EINVAL), (dict(type=-1), EUNSUP), (dict(type=3), EUNSUP), (dict(ko=None), EINVAL), (dict(vo=None), EINVAL),
    (dict(ko=MIS), EINVAL), (dict(vo=MIS), EINVAL), (dict(T=1 << 29, n_kv_heads=8), EINVAL), (dict(T=0, ko=None, vo=None), OK)])
def test_read_argument_errors(kw, code):
    assert _read(**dict(kw)) == code


def test_python_refusals_without_a_gpu():
    import torch
    q = torch.zeros(4, 2, 64).bfloat16()
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        ltk.attend_prompt(q, q, q, cu)
    for bad, err in ((q.float(), TypeError), (q[0], ValueError), (None, TypeError)):
        with pytest.raises(err):
            ltk.attend_prompt(bad, q, q, cu)
