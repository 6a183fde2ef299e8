"""The sparse step as a whole: what a refused call leaves behind."""
import pytest

from tests.attend_ref import make_batch, make_cache
from tests.test_gpu_attend import _dev, _gen

pytestmark = pytest.mark.gpu


def _step(T=3, L=50, D=64):
    import torch
    g = _gen(75)
    table, _, n, pages = make_batch(g, [T], [L], 16)
    r = lambda *s: torch.randn(*s, generator=g)
    q, k, v = r(T, 4, D).bfloat16(), r(T, 2, D).bfloat16(), r(T, 2, D).bfloat16()
    cache = _dev(*make_cache(g, pages, 2, 16, D))
    a = dict(zip(("q", "k", "v", "page_table", "kv_len", "index_q", "index_k", "index_w"),
                 _dev(q, k, v, table, n, r(T, 4, D).bfloat16(), r(L, D).bfloat16(), torch.rand(T, 4, generator=g))))
    return dict(a, cache=cache, topk=8)


def test_a_refused_step_leaves_the_cache(lib):
    import torch
    a = _step()
    before = [t.clone() for t in a["cache"]]
    wrong = [dict(topk=0), dict(topk=65537), dict(index_w=a["index_w"][:, :3].contiguous()), dict(index_q=a["index_q"].half()),
             dict(index_k=a["index_k"][:, ::2]), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=3e38),
             dict(out=torch.empty_like(a["q"]).float()), dict(out=torch.empty_like(a["q"])[:2]),
             dict(out=torch.empty(a["q"].shape, dtype=torch.bfloat16)), dict(q=a["q"][:, :3].contiguous()),
             dict(v=a["v"][:2].contiguous()), dict(inv_freq=torch.ones(8, device="cuda")), dict(index_q_scale=torch.ones(3, device="cuda"))]
    for w in wrong:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            lib.sparse_step(**{**a, **w})
        for x, y in zip(before, a["cache"]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), w.keys()
    out = torch.empty_like(a["q"])
    got, idx = lib.sparse_step(**a, out=out, scale=0.1)
    assert got is out and idx.shape == (3, 8)
    assert not all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, a["cache"]))
