"""Attention over 16-bit prompts and its gradient against 64 bits."""
import math

import pytest

from tests.prompt_ref import check, lens_to_cu, make, ref

pytestmark = pytest.mark.gpu


def _run(lib, q, k, v, dout, cu, cu_k, scale=None, window=0):
    import torch
    dev = [x.cuda().requires_grad_() for x in (q, k, v)]
    dcu, dck = cu.cuda(), None if cu_k is None else cu_k.cuda()
    out, lse = lib.attend_prompt(*dev, dcu, dck, scale=scale, window=window, return_lse=True)
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(out, dev, dout.cuda())))
    with torch.no_grad():   # the same without a graph
        again = lib.attend_prompt(*dev, dcu, dck, scale=scale, window=window)
    assert torch.equal(again, out) and out.requires_grad and not lse.requires_grad
    return dict(got, out=out, lse=lse)


def _case(lib, rows, keys, Hq, Hkv, D, dtype, seed, window=0, scale=None, spread=1.0, before=0, behind=0):
    import torch
    dt = getattr(torch, dtype)
    q, k, v, dout = make(seed, rows, keys or rows, Hq, Hkv, D, dt, spread, before, behind)
    if behind or before:   # what lies outside every sequence may be anything
        for x in (q, k, v, dout):
            x[:before] = math.nan
            x[x.shape[0] - behind:] = math.nan if behind else 0
    cu = lens_to_cu(rows, before)
    cu_k = lens_to_cu(keys, before) if keys else None
    got = _run(lib, q, k, v, dout, cu, cu_k, scale, window)
    want = ref(q, k, v, cu, cu if cu_k is None else cu_k, scale or D ** -0.5, window, dout)
    for name, w in want.items():
        if name != "lse":
            w = (w[0], w[1])
        check(name, got[name], w)
    return got


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (6, 2), (7, 1), (16, 2)])
def test_lengths(lib, Hq, Hkv, D, dtype):
    _case(lib, [1, 0, 63, 64, 65, 2, 130], None, Hq, Hkv, D, dtype, 11 + D + Hq)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 257, 600])
@pytest.mark.parametrize("D", [64, 128])
def test_one_prompt(lib, n, D):
    _case(lib, [n], None, 3, 3, D, "bfloat16", n)


@pytest.mark.parametrize("rows,keys", [
    ([1], [500]), ([5], [64]), ([70, 3], [200, 3]), ([40, 1, 9], [0, 1, 200]),      # no keys at all; a history
    ([64, 30], [10, 130]),                                                       # the first rows see nothing
    ([1, 1, 1], [700, 1, 65]), ([0, 0], [50, 3]), ([0, 4], [0, 0]),
])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 17])
def test_histories_and_empty_rows(lib, rows, keys, D, window):
    got = _case(lib, rows, keys, 4, 2, D, "bfloat16", 3 + D, window=window)
    assert not any(bool(x.isnan().any()) for x in got.values())


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(2, 2, 64, "float16"), (10, 2, 128, "bfloat16")])
def test_windows(lib, window, Hq, Hkv, D, dtype):
    _case(lib, [300, 77, 1], None, Hq, Hkv, D, dtype, window % 1000, window=window)


@pytest.mark.parametrize("before,behind", [(0, 5), (3, 0), (130, 150)])
@pytest.mark.parametrize("keys", [None, [10, 90]])
def test_rows_outside_every_sequence(lib, before, behind, keys):
    import torch
    got = _case(lib, [40, 70], keys, 4, 2, 64, "bfloat16", 5, before=before, behind=behind)
    for name, x in got.items():
        want = -math.inf if name == "lse" else 0
        rest = torch.cat([x[:before], x[x.shape[0] - behind:] if behind else x[:0]])
        assert bool((rest == want).all()), name


@pytest.mark.parametrize("n_seq", [0, 1])
def test_no_sequence_or_an_empty_one(lib, n_seq):
    import torch
    q, k, v, dout = make(1, [9], [9], 4, 2, 64, torch.bfloat16)
    got = _run(lib, q, k, v, dout, torch.zeros(n_seq + 1, dtype=torch.int32), None)
    assert all(bool((x == (-math.inf if n == "lse" else 0)).all()) for n, x in got.items())
    e = [x[:0] for x in (q, k, v, dout)]
    got = _run(lib, *e, torch.zeros(n_seq + 1, dtype=torch.int32), None)
    assert got["out"].shape == (0, 4, 64) and got["dk"].shape == (0, 2, 64)


@pytest.mark.parametrize("scale", [0.0, -0.125, 0.5, 3.0])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_scales(lib, scale, dtype):
    import torch
    q, k, v, dout = make(8, [150], [150], 4, 2, 64, getattr(torch, dtype))
    cu = lens_to_cu([150])
    got = _run(lib, q, k, v, dout, cu, None, scale)
    for name, w in ref(q, k, v, cu, cu, scale, 0, dout).items():
        check(name, got[name], w)


@pytest.mark.parametrize("D", [64, 128])
def test_rising_scores_move_the_reference(lib, D):
    """Each key's score passes those before it by more than the slack of the running reference."""
    import torch
    n = 300
    q, k, v, dout = make(21, [n], [n], 2, 1, D, torch.bfloat16)
    q[:] = 1.0
    k[:] = (torch.arange(n)[:, None, None] // 4 * (12.0 / D ** 0.5)).to(k.dtype)
    cu = lens_to_cu([n])
    got = _run(lib, q, k, v, dout, cu, None)
    for name, w in ref(q, k, v, cu, cu, D ** -0.5, 0, dout).items():
        check(name, got[name], w)


@pytest.mark.parametrize("layout", ["fused", "heads first", "wide", "broadcast", "odd", "misaligned", "last"])
@pytest.mark.parametrize("D", [64, 128])
def test_strides(lib, layout, D):
    import torch
    rows, Hq, Hkv = [45, 100], 6, 2
    T = sum(rows)
    q, k, v, dout = [x.cuda() for x in make(31, rows, rows, Hq, Hkv, D, torch.bfloat16)]
    cu = lens_to_cu(rows)

    def lay(x):
        n, h, d = x.shape
        if layout == "fused":
            y = torch.zeros(n, h + 5, d, device="cuda", dtype=x.dtype)[:, 2:2 + h]
        elif layout == "heads first":
            y = torch.zeros(h, n, d, device="cuda", dtype=x.dtype).transpose(0, 1)
        elif layout == "wide":
            y = torch.zeros(2 * n, h, d + 8, device="cuda", dtype=x.dtype)[::2, :, :d]
        elif layout == "odd":
            y = torch.zeros(n, h, d + 3, device="cuda", dtype=x.dtype)[:, :, :d]
        elif layout == "misaligned":
            y = torch.zeros(n * h * d + 1, device="cuda", dtype=x.dtype)[1:].view(n, h, d)
        elif layout == "last":
            y = torch.zeros(n, d, h, device="cuda", dtype=x.dtype).transpose(1, 2)
        else:
            return x[:1, :1].expand(n, h, d)
        return y.copy_(x)
    args = [lay(x) for x in (q, k, v)]
    leaves = [x.detach().requires_grad_() for x in args]
    out = lib.attend_prompt(*leaves, cu.cuda())
    g = torch.autograd.grad(out, leaves, lay(dout))
    want = ref(*[x.cpu() for x in args], cu, cu, D ** -0.5, 0, lay(dout).cpu())
    for name, x in zip(("out", "dq", "dk", "dv"), (out,) + g):
        check(name, x, want[name])


def test_cut_work_is_joined(lib):
    """Few units over many keys (and few keys' rows): parts of both passes."""
    _case(lib, [3], [2500], 2, 1, 128, "bfloat16", 41)
    _case(lib, [900], None, 1, 1, 64, "float16", 42)
    _case(lib, [200, 700], [1500, 700], 5, 1, 64, "bfloat16", 43)
    _case(lib, [900], None, 3, 1, 128, "bfloat16", 44, window=300)


def test_many_sequences(lib):
    rows = [(7 * i) % 23 for i in range(700)]
    _case(lib, rows, None, 2, 1, 64, "bfloat16", 51)


def test_offsets_past_the_tensors_and_out_of_order(lib):
    """Whatever cu holds, nothing outside the tensors is touched; ordered sequences keep their results."""
    import torch
    q, k, v, dout = [x.cuda() for x in make(61, [50, 60], [50, 60], 4, 2, 64, torch.bfloat16)]
    with torch.no_grad():
        want = lib.attend_prompt(q, k, v, lens_to_cu([50, 60]).cuda())
        got = lib.attend_prompt(q, k, v, torch.tensor([0, 50, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
        assert torch.equal(got, want)
        for bad in ([-5, 30, 10, 110], [110, 0, 50, -(2 ** 31)], [2 ** 31 - 1, 2 ** 31 - 1, 0, 7]):
            lib.attend_prompt(q, k, v, torch.tensor(bad, dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()


def test_same_bits_again(lib):
    import torch
    q, k, v, dout = make(71, [300, 200], [300, 200], 8, 2, 128, torch.bfloat16)
    cu = lens_to_cu([300, 200])
    first = _run(lib, q, k, v, dout, cu, None)
    for _ in range(3):
        for name, x in _run(lib, q, k, v, dout, cu, None).items():
            assert torch.equal(x, first[name]), name


def test_gradient_against_differences(lib):
    """Inner products of the gradients with directions against central differences of the 64-bit form."""
    import torch
    rows, keys = [20, 33], [50, 33]
    q, k, v, dout = make(81, rows, keys, 4, 2, 64, torch.float16)
    cu, ck = lens_to_cu(rows), lens_to_cu(keys)
    got = _run(lib, q, k, v, dout, cu, ck)
    want = ref(q, k, v, cu, ck, 0.125, 0, dout)
    x = dict(q=q.double(), k=k.double(), v=v.double())

    def loss(**moved):
        t = dict(x, **moved)
        total = 0.0
        for b in range(2):
            for h in range(4):
                z = t["q"][cu[b]:cu[b + 1], h] @ t["k"][ck[b]:ck[b + 1], h // 2].T * 0.125
                n, m = z.shape
                z = z.masked_fill(torch.arange(m) > m - n + torch.arange(n)[:, None], -math.inf)
                total += float((torch.softmax(z, -1) @ t["v"][ck[b]:ck[b + 1], h // 2] * dout[cu[b]:cu[b + 1], h].double()).sum())
        return total
    for name in ("q", "k", "v"):
        d = torch.randn(x[name].shape, generator=torch.Generator().manual_seed(9), dtype=torch.float64)
        diff = lambda h: (loss(**{name: x[name] + h * d}) - loss(**{name: x[name] - h * d})) / (2 * h)
        h = 2.0 ** -12
        slope, curve = diff(h), abs(diff(h) - diff(2 * h))       # the difference's own error is below `curve`
        tol = float((want["d" + name][1] * d.abs()).sum())
        assert abs(float((got["d" + name].cpu().double() * d).sum()) - slope) <= tol + curve + 1e-9


def test_only_some_gradients(lib):
    import torch
    q, k, v, dout = [x.cuda() for x in make(91, [80], [80], 4, 2, 64, torch.bfloat16)]
    cu = lens_to_cu([80]).cuda()
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    full = torch.autograd.grad(lib.attend_prompt(*leaves, cu), leaves, dout)
    for i in range(3):
        args = [q, k, v]
        args[i] = leaves[i]
        (g,) = torch.autograd.grad(lib.attend_prompt(*args, cu), [leaves[i]], dout)
        assert torch.equal(g, full[i])
    # heads shared by expanding one: their sum
    one = k[:, :1].clone().requires_grad_()
    (g,) = torch.autograd.grad(lib.attend_prompt(q, one.expand(80, 2, 64), v, cu), [one], dout)
    args = [q, k[:, :1].expand(80, 2, 64).contiguous().requires_grad_(), v]
    (w,) = torch.autograd.grad(lib.attend_prompt(*args, cu), [args[1]], dout)
    assert torch.allclose(g.float(), w.float().sum(1, keepdim=True), rtol=2.0 ** -7, atol=1e-3)


def test_refusals_of_autograd(lib):
    import torch
    import torch.autograd.forward_ad as fwd
    q, k, v, dout = [x.cuda() for x in make(95, [20], [20], 2, 1, 64, torch.bfloat16)]
    cu = lens_to_cu([20]).cuda()
    leaf = q.clone().requires_grad_()
    out = lib.attend_prompt(leaf, k, v, cu)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(out, leaf, dout, create_graph=True)
    out = lib.attend_prompt(leaf, k, v, cu)
    with torch.no_grad():
        out.mul_(2)              # the backward pass reads what the forward pass returned
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out, leaf, dout)
    with fwd.dual_level(), pytest.raises(RuntimeError, match="tangent"):
        lib.attend_prompt(fwd.make_dual(q, torch.ones_like(q)), k, v, cu)
    with torch.inference_mode():
        assert torch.equal(lib.attend_prompt(q.clone(), k, v, cu), lib.attend_prompt(q, k, v, cu))


def test_training_moves_weights_as_the_plain_form_does(lib):
    """q, k and v as slices of one projection of packed sequences; the projection's gradient against 64 bits."""
    import torch
    rows, Hq, Hkv, D, W = [33, 20, 70], 4, 2, 64, 96
    g = torch.Generator().manual_seed(3)
    x = torch.randn(sum(rows), W, generator=g).bfloat16()
    w = (torch.randn(W, (Hq + 2 * Hkv) * D, generator=g) / W ** 0.5).bfloat16()
    cu = lens_to_cu(rows)
    wd = w.cuda().requires_grad_()
    y = (x.cuda() @ wd).view(-1, Hq + 2 * Hkv, D)
    q, k, v = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    out = lib.attend_prompt(q, k, v, cu.cuda())
    dout = torch.randn(out.shape, generator=g).bfloat16()
    out.backward(dout.cuda())
    want = ref(q.detach().cpu(), k.detach().cpu(), v.detach().cpu(), cu, cu, D ** -0.5, 0, dout)
    dy, ty = (torch.cat([want[n][i] for n in ("dq", "dk", "dv")], 1).reshape(sum(rows), -1) for i in (0, 1))
    # the sum of gradients in bf16 (each rounded once more by the slices' join), then an fp32-accumulated product
    val = x.double().T @ dy
    tol = x.double().abs().T @ (ty + 2.0 ** -7 * dy.abs()) + 2.0 ** -8 * val.abs()
    check("weights", wd.grad, (val, tol * 1.01))


def test_captured(lib):
    """Forward and backward in one captured graph, replayed with new inputs between eager work."""
    import torch
    rows = [100, 60]
    cu = lens_to_cu(rows).cuda()
    sets = [[x.cuda() for x in make(s, rows, rows, 8, 2, 128, torch.bfloat16)] for s in (1, 2, 3)]
    buf = [x.clone() for x in sets[0]]
    leaves = [x.requires_grad_() for x in buf[:3]]

    def step():
        out = lib.attend_prompt(*leaves, cu)
        return (out.detach(),) + torch.autograd.grad(out, leaves, buf[3])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for data in sets + sets[:1]:
        with torch.no_grad():
            for b, x in zip(buf, data):
                b.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        held = [x.clone() for x in got]
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_capture_beside_an_eager_graph_of_the_same_leaf_is_refused(lib):
    import torch
    q, k, v, dout = [x.cuda() for x in make(7, [30], [30], 2, 1, 64, torch.bfloat16)]
    cu = lens_to_cu([30]).cuda()
    q.requires_grad_()
    alive = lib.attend_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(graph):
            lib.attend_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="still alive"):   # .. also where the call's inputs are made of the leaf
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            lib.attend_prompt((q * 2)[:, :], k, v, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):           # (no backward pass can follow)
        out = lib.attend_prompt(q, k, v, cu)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, alive)
    (g,) = torch.autograd.grad(alive, q, dout)
    assert bool(g.isfinite().all())


def test_streams(lib):
    """A call on a side stream reads what was enqueued there before it."""
    import torch
    rows = [200, 150]
    q, k, v, dout = [x.cuda() for x in make(17, rows, rows, 8, 2, 64, torch.bfloat16)]
    cu = lens_to_cu(rows).cuda()
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    out = lib.attend_prompt(*leaves, cu)
    want = (out.detach(),) + torch.autograd.grad(out, leaves, dout)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mine = [torch.zeros_like(x) for x in (q, k, v)]
        for _ in range(20):
            for m, x in zip(mine, (q, k, v)):
                m.copy_(x)
        mine = [m.requires_grad_() for m in mine]
        out = lib.attend_prompt(*mine, cu)
        got = (out.detach(),) + torch.autograd.grad(out, mine, dout)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [2, 5, 8, 12, 16, 24, 40])
def test_groups(lib, G, D):
    """Heads that fill copies of rows evenly and such that do not."""
    _case(lib, [90, 33], [90, 50], 2 * G, 2, D, "bfloat16", 100 + G)


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (6, 2)])
def test_long_sequences_cut_in_both_passes(lib, Hq, Hkv):
    """Lengths at which units are cut in parts by rule, whole parts and rests, beside short sequences."""
    _case(lib, [1700, 65, 400], None, Hq, Hkv, 64, "bfloat16", 111)
    _case(lib, [300, 20], [2300, 1000], Hq, Hkv, 128, "bfloat16", 112)


def test_offsets_past_32_bits(lib):
    """The last sequence of tensors of more than 2^31 elements gets what it gets alone."""
    import torch
    T0, n, H, D, w = (1 << 17) - 100, 300, 128, 128, 64
    T = T0 + n
    small = [x.cuda() for x in make(120, [n], [n], H, 4, D, torch.bfloat16)]
    q, dout = (torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(T, 4, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert q.numel() > 1 << 31
    for x, y in zip((q, k, v, dout), small):
        x[T0:] = y
    leaves = [x.requires_grad_() for x in (q, k, v)]
    cu = torch.tensor([0, T0, T], dtype=torch.int32, device="cuda")
    out = lib.attend_prompt(*leaves, cu, window=w)
    got = (out.detach(),) + torch.autograd.grad(out, leaves, dout)
    mine = [x.clone().requires_grad_() for x in small[:3]]
    out = lib.attend_prompt(*mine, cu[:2].clone().fill_(0).index_fill_(0, torch.tensor([1], device="cuda"), n), window=w)
    want = (out.detach(),) + torch.autograd.grad(out, mine, small[3])
    # (units of the two calls may be cut differently: sums in another order, then one rounding)
    for a, b in zip(got, want):
        assert torch.allclose(a[T0:].float(), b.float(), rtol=2.0 ** -6, atol=2.0 ** -6)
        assert bool((a[:T0] == 0).all())


def test_on_another_device_context(lib):
    """The call runs on its tensors' device and stream whatever thread makes it."""
    import threading
    import torch
    q, k, v, dout = [x.cuda() for x in make(130, [60], [60], 4, 2, 64, torch.bfloat16)]
    cu = lens_to_cu([60]).cuda()
    leaves = [x.requires_grad_() for x in (q, k, v)]
    out = lib.attend_prompt(*leaves, cu)
    want = (out.detach(),) + torch.autograd.grad(out, leaves, dout)
    res = {}

    def work(i):
        for _ in range(10):
            o = lib.attend_prompt(*leaves, cu)
            res[i] = (o.detach(),) + torch.autograd.grad(o, leaves, dout)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    [t.start() for t in threads], [t.join() for t in threads]
    torch.cuda.synchronize()
    assert len(res) == 3 and all(torch.equal(a, b) for r in res.values() for a, b in zip(r, want))


def test_captured_with_a_leaf_used_twice(lib):
    """The second call finds the leaf held by the captured graph itself: no other stream waits."""
    import torch
    rows = [70, 41]
    cu = lens_to_cu(rows).cuda()
    q, k, v, dout = [x.cuda() for x in make(140, rows, rows, 4, 2, 64, torch.bfloat16)]
    leaves = [x.requires_grad_() for x in (q, k, v)]

    def step():
        a = lib.attend_prompt(*leaves, cu)
        b = lib.attend_prompt(a, k, v, cu)
        return (b.detach(),) + torch.autograd.grad(b, leaves, dout)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        with torch.no_grad():
            q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        held = [x.clone() for x in got]
        assert all(torch.equal(x, y) for x, y in zip(held, step()))


def test_captured_while_the_warm_up_on_a_side_stream_lives(lib):
    import torch
    rows = [70, 41]
    cu = lens_to_cu(rows).cuda()
    q, k, v, dout = [x.cuda() for x in make(141, rows, rows, 4, 2, 64, torch.bfloat16)]
    leaves = [x.requires_grad_() for x in (q, k, v)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        alive = lib.attend_prompt(*leaves, cu)
        want = torch.autograd.grad(alive, leaves, dout, retain_graph=True)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(lib.attend_prompt(*leaves, cu), leaves, dout)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and alive.grad_fn is not None


def test_more_sequences_than_one_look_covers(lib):
    """4,300 sequences, most of them empty or of one row: found over two levels of looks."""
    rows = [(i * 7) % 3 if i % 2 else 0 for i in range(4300)]
    _case(lib, rows, None, 1, 1, 64, "bfloat16", 151)
