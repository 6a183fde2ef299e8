"""What cu, cu_k, groups and lengths hold is data: outputs and workspaces between guarded bytes, inputs as they were."""
import ctypes

import pytest

from tests.test_attend_abi import P
from tests.test_gpu_shared import shared_case
from tests.test_prompt_abi import CPrompt, CRows

pytestmark = pytest.mark.gpu

GUARD, MARK = 1 << 16, 0xA5
_FAR = (2 ** 31 - 1, -(2 ** 31))


class Guarded:
    """Buffers of one allocation, each between GUARD marked bytes."""

    def __init__(self, sizes):
        import torch
        self.at, end = {}, GUARD
        for name, n in sizes.items():
            self.at[name] = (end, n)
            end += (n + 255) // 256 * 256 + GUARD
        self.all = torch.full((end,), MARK, dtype=torch.uint8, device="cuda")
        self.outside = torch.ones(end, dtype=torch.bool, device="cuda")
        for a, n in self.at.values():
            self.outside[a:a + n] = False

    def ptr(self, name):
        return self.all.data_ptr() + self.at[name][0]

    def bytes(self, name):
        a, n = self.at[name]
        return self.all[a:a + n]

    def check(self):
        import torch
        torch.cuda.synchronize()
        assert bool((self.all[self.outside] == MARK).all())


def _offsets(seed, n, most):
    """n + 1 offsets in no order: inside, at the ends of and outside [0, most], and of 32 bits."""
    import torch
    g = torch.Generator().manual_seed(seed)
    inside = torch.randint(-5, most + 6, (n + 1,), generator=g)
    pick = torch.randint(0, 8, (n + 1,), generator=g)
    for i, x in enumerate((0, most) + _FAR):
        inside[pick == i] = x
    return inside.int()


@pytest.mark.parametrize("dtype,D,Hq,Hkv,T,S", [
    ("bfloat16", 64, 4, 2, 110, 110), ("float16", 128, 3, 1, 300, 700), ("bfloat16", 128, 16, 2, 77, 4000),
    ("bfloat16", 64, 2, 2, 2000, 2000), ("float16", 64, 1, 1, 5000, 5000)])
@pytest.mark.parametrize("n_seq", [1, 3, 70])
def test_offsets_in_no_order(lib, dtype, D, Hq, Hkv, T, S, n_seq):
    import torch
    L = lib.library()
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(T + n_seq)
    shapes = dict(q=(T, Hq, D), k=(S, Hkv, D), v=(S, Hkv, D), dout=(T, Hq, D))
    host = {x: torch.randn(s, generator=g).to(dt) for x, s in shapes.items()}
    sizes = {x: t.numel() * 2 for x, t in host.items()}
    sizes.update(out=T * Hq * D * 2, rest=T * Hq * D * 2, lse=T * Hq * 4, dq=T * Hq * D * 2, dk=S * Hkv * D * 2, dv=S * Hkv * D * 2)
    f = L.litetopk_attend_prompt_workspace_bytes
    f.restype, f.argtypes = ctypes.c_size_t, [ctypes.c_void_p, ctypes.c_int32]
    rc = L.litetopk_attend_prompt
    rc.restype = ctypes.c_int
    rc.argtypes = [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]
    rb = L.litetopk_attend_prompt_backward
    rb.restype = ctypes.c_int
    rb.argtypes = [ctypes.c_void_p] * 12 + [ctypes.c_size_t, ctypes.c_void_p]
    stream = torch.cuda.current_stream().cuda_stream
    for window in (0, 33):
        p = CPrompt(P, P, n_seq, T, S, Hq, Hkv, D, 0 if dtype == "bfloat16" else 1, D ** -0.5, window)
        ws = [f(ctypes.byref(p), back) for back in (0, 1)]
        buf = Guarded(dict(sizes, ws=max(ws)))
        for x, t in host.items():
            buf.bytes(x).copy_(t.reshape(-1).view(torch.uint8))
        rows = {x: CRows(buf.ptr(x), s[1] * D, D) for x, s in shapes.items()}
        r = {x: ctypes.byref(y) for x, y in rows.items()}
        for seed in range(4):
            cu, cu_k = _offsets(seed, n_seq, T).cuda(), _offsets(100 + seed, n_seq, S).cuda()
            if seed == 0:                            # (and in order, all rows and keys in sequences)
                cu, cu_k = (x.clamp(0, n).sort()[0] for x, n in ((cu, T), (cu_k, S)))
                cu[0], cu[-1], cu_k[0], cu_k[-1] = 0, T, 0, S
            own = S == T and seed % 2 == 0
            p.cu, p.cu_k = cu.data_ptr(), None if own else cu_k.data_ptr()
            buf.bytes("ws").fill_(0xFF)              # (NaN)
            assert rc(ctypes.byref(p), r["q"], r["k"], r["v"], buf.ptr("out"), buf.ptr("rest"), buf.ptr("lse"), buf.ptr("ws"),
                      ws[0], stream) == 0
            buf.check()
            for dq, dk, dv in (("dq", "dk", "dv"), (None, "dk", "dv"), ("dq", None, None)):
                ptr = [None if x is None else buf.ptr(x) for x in (dq, dk, dv)]
                assert rb(ctypes.byref(p), r["q"], r["k"], r["v"], buf.ptr("out"), buf.ptr("rest"), buf.ptr("lse"), r["dout"],
                          *ptr, buf.ptr("ws"), ws[1], stream) == 0
                buf.check()
        for x, t in host.items():
            assert torch.equal(buf.bytes(x).cpu().view(dt).view(t.shape), t)


@pytest.mark.parametrize("rows,Hkv,G", [(1, 2, 4), (40, 1, 8)])       # both kernels
def test_groups_in_no_order(lib, rows, Hkv, G):
    import torch
    tokens = [rows + 900, rows + 1200, rows + 300, rows + 64]
    q, cache, table, cu, kv_len, bounds, lens = shared_case(21, [(256, [(rows, t) for t in tokens])], Hkv, G, 16, 64)
    T, Hq = q.shape[:2]
    d, args = [x.cuda() for x in cache], [x.cuda() for x in (table, cu, kv_len)]
    kept = [x.clone() for x in d]
    for n_group in (1, 2, 9):
        need = lib.attend_shared_workspace_bytes(T, Hq, Hkv, 64, 4, n_group, table.shape[1] * 16)
        buf = Guarded(dict(out=T * Hq * 64 * 2, ws=need))
        out = buf.bytes("out").view(torch.bfloat16).view(T, Hq, 64)
        for seed in range(6):
            groups = _offsets(seed, n_group, 4).cuda()
            shared = _offsets(50 + seed, n_group - 1, table.shape[1] * 16).cuda()
            buf.bytes("ws").fill_(0xFF)
            lib.attend_shared(q.cuda(), d, *args, groups, shared, out=out, workspace=buf.bytes("ws"))
            buf.check()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(d, kept))
