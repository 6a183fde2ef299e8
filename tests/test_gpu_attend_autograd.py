"""The paged cache's operators under autograd: they are forward only."""
import pytest

from tests.test_gpu_attend import _attend_case, _dev, _lists, _gen

pytestmark = pytest.mark.gpu


def _calls(lib):
    """Per entry: its name, and the call with q (kv_append: k, v and q) taken from a dict."""
    import torch
    cache, table, cu, n, q = _attend_case([6], [90], 2, 4, 16, 64, 85)
    dc, (dt, dcu, dn) = _dev(*cache), _dev(table, cu, n)
    idx = _lists(_gen(86), [6], [90], 20).cuda()
    sh, m, ln = lib.dsa_pack(idx, 90, 3)
    k = torch.randn(6, 2, 64, generator=_gen(87)).bfloat16()
    t = dict(q=q.cuda(), k=k.cuda(), v=k.cuda(), k_scale=dc[2], v_scale=dc[3], out=torch.empty_like(q).cuda(),
             inv_freq=torch.ones(32, dtype=torch.float64, device="cuda"))
    c = lambda x: (dc[0], dc[1], x["k_scale"], x["v_scale"])
    return t, {
        "kv_append": (("k", "v", "q", "k_scale", "v_scale", "inv_freq", "out"), lambda x: lib.kv_append(
            x["k"], x["v"], c(x), dt, dcu, dn, x["inv_freq"], x["q"], q_out=x["out"])),
        "attend": (("q", "k_scale", "v_scale", "out"), lambda x: lib.attend(x["q"], c(x), dt, dcu, dn, out=x["out"])),
        "attend_selected": (("q", "out"), lambda x: lib.attend_selected(x["q"], c(x), dt, dcu, dn, idx, out=x["out"])),
        "attend_packed": (("q", "out"), lambda x: lib.attend_packed(x["q"], c(x), dt, dn, sh, m, ln, 3, out=x["out"])),
    }


@pytest.mark.parametrize("entry", ["kv_append", "attend", "attend_selected", "attend_packed"])
def test_tensors_that_autograd_follows_are_refused(lib, entry):
    import torch
    import torch.autograd.forward_ad as fwd
    t, calls = _calls(lib)
    names, call = calls[entry]
    before = [x.clone() for x in t.values()]
    for name in names:
        x = dict(t)
        x[name] = t[name].clone().requires_grad_()
        with pytest.raises(RuntimeError, match="requires grad"):
            call(x)
        with fwd.dual_level():
            x[name] = fwd.make_dual(t[name].clone(), torch.ones_like(t[name]))
            with pytest.raises(RuntimeError, match="tangent"), torch.no_grad():
                call(x)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, t.values()))   # nothing ran
    want = call(t).clone()
    with torch.no_grad():      # a followed tensor as an input is welcome here
        got = call({**t, "q": t["q"].clone().requires_grad_()})
    assert torch.equal(got, want) and not got.requires_grad
    with torch.inference_mode():
        assert torch.equal(call({**t, "q": t["q"].clone()}), want)


def test_what_is_written_in_place_counts_versions(lib):
    """The cache and given outputs, so that a backward pass which saved one of them before notices."""
    import torch
    t, calls = _calls(lib)
    versions = lambda: {name: x._version for name, x in t.items()}
    v0 = versions()
    calls["attend"][1](t)
    v1 = versions()
    assert v1["out"] > v0["out"] and all(v1[n] == v0[n] for n in t if n != "out")
    x = torch.ones(1, device="cuda", requires_grad=True)
    y = (x * t["k_scale"]).sum()                     # saves the scales
    calls["kv_append"][1](t)
    v2 = versions()
    assert all(v2[n] > v1[n] for n in ("out", "k_scale", "v_scale")) and v2["q"] == v1["q"] and v2["k"] == v1["k"]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    for entry in ("attend_selected", "attend_packed"):
        before = t["out"]._version
        calls[entry][1](t)
        assert t["out"]._version > before
    with torch.inference_mode():                     # no versions there
        inf = {n: a.clone() for n, a in t.items()}
        for _, call in calls.values():
            call(inf)
    for _, call in calls.values():
        call(inf)                                    # .. nor outside it, of its tensors


def test_a_cache_list_emptied_while_the_call_reads_its_arguments(lib):
    """The call holds the tensors that it took from the list."""
    import torch
    cache, table, cu, n, q = _attend_case([2], [90], 2, 4, 16, 64, 88)
    a = _dev(table, cu, n)
    want = lib.attend(q.cuda(), _dev(*cache), *a, scale=0.25)
    held = list(_dev(*cache))

    class Scale:
        def __float__(self):
            held.clear()
            self.other = [torch.full_like(t.cuda().view(torch.uint8), 0x7F) for t in cache]   # takes what was freed
            return 0.25

    assert torch.equal(lib.attend(q.cuda(), held, *a, scale=Scale()), want) and not held


@pytest.mark.parametrize("at", [0, 1, 2, 3])
@pytest.mark.parametrize("what", [None, 3, "k", [1.0]])
def test_a_cache_entry_that_is_no_tensor_is_refused(lib, at, what):
    cache, table, cu, n, q = _attend_case([2], [90], 2, 4, 16, 64, 88)
    c = list(_dev(*cache))
    c[at] = what
    for wrong in (c, tuple(c)):
        with pytest.raises(TypeError, match="must be a tensor"):
            lib.attend(q.cuda(), wrong, *_dev(table, cu, n))
