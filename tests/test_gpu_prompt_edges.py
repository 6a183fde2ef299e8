"""attend_prompt where its inputs' strides, sizes and weights are at their ends."""
import pytest

from tests.prompt_ref import check, lens_to_cu, make, ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,strides", [
    ((1, 2, 64), (7, 64, 1)), ((40, 1, 64), (64, 5, 1)), ((1, 1, 128), (3, 5, 1)), ((1, 2, 64), (1 << 24, 64, 1)),
])
def test_any_stride_of_a_dimension_of_one(lib, shape, strides):
    """Tensors off 16 bytes are copied, whatever the strides are that their dimensions of size 1 carry."""
    import torch
    n, h, d = shape
    data = [x.cuda() for x in make(3, [n], [n], h, h, d, torch.bfloat16)]
    cu = lens_to_cu([n])
    want = ref(*[x.cpu() for x in data[:3]], cu, cu, d ** -0.5, 0, data[3].cpu())

    def lay(x):
        flat = torch.zeros(x.numel() + 8, device="cuda", dtype=x.dtype)
        return flat.as_strided(shape, strides, 1).copy_(x)
    leaves = [lay(x).detach().requires_grad_() for x in data[:3]]
    assert leaves[0].stride() == strides and leaves[0].data_ptr() % 16 != 0
    out = lib.attend_prompt(*leaves, cu.cuda())
    got = (out,) + torch.autograd.grad(out, leaves, lay(data[3]))
    for name, x in zip(("out", "dq", "dk", "dv"), got):
        check(name, x, want[name])


def test_a_head_dim_past_32_bits_is_refused(lib):
    import torch
    q = torch.empty(0, 1, (1 << 32) + 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="too large"):
        lib.attend_prompt(q, q, q, cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("n", [250, 900])
def test_gradients_of_values_with_small_weights_in_fp16(lib, n, G, D):
    """Weights of 2^-30 to 2^-24, beside one of about 1, under a scaled loss: dv to fp16's own precision.

    The bounds of prompt_ref, but for its 2^-25 of a weight: dv_s = sum_i P_is dout_i is off by
      u |dv_s| + sum_i (P_is (u + 2 E + N 2^-23) + 2^-39) |dout_i| + 2^-25
    over the N rows and heads, where 2^-39 is half a step of fp16 below 2^-14 for weights held 2^14 times
    their size, and 2^-25 that of the result."""
    import torch
    m, u = n + 70, 2.0 ** -11
    g = torch.Generator().manual_seed(n + G + D)
    q, k = torch.zeros(n, G, D, dtype=torch.float16), torch.zeros(m, 1, D, dtype=torch.float16)
    q[:, :, 0] = 1
    k[1:, 0, 0] = (-17.0 - 3.5 * torch.rand(m - 1, generator=g)).half()
    v = torch.randn(m, 1, D, generator=g).half()
    dout = (2.0 ** 12 * torch.randn(n, G, D, generator=g)).half()
    cu, ck = lens_to_cu([n]), lens_to_cu([m])
    leaves = [x.cuda().requires_grad_() for x in (q, k, v)]
    out = lib.attend_prompt(*leaves, cu.cuda(), ck.cuda(), scale=1.0)
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(out, leaves, dout.cuda())))
    want = ref(q, k, v, cu, ck, 1.0, 0, dout)
    for name in ("dq", "dk"):
        check(name, got[name], want[name])
    x = k[:, 0, 0].double().expand(n, m).masked_fill(torch.arange(m) > m - n + torch.arange(n)[:, None], -torch.inf)
    P = torch.softmax(x, -1)
    assert float(P[:, 1:].max()) < 2.0 ** -24 and float(P[-1, 1:].min()) > 2.0 ** -30
    lse = torch.logsumexp(x, -1).abs().max()
    E = (D + 8) * 2.0 ** -24 * (2 * 20.5 + float(lse)) + 2.0 ** -22
    val = torch.zeros(m, D, dtype=torch.float64)
    size = torch.zeros_like(val)
    for h in range(G):
        val += P.T @ dout[:, h].double()
        size += (P * (u + 2 * E + n * G * 2.0 ** -23) + 2.0 ** -39 * (P > 0)).T @ dout[:, h].double().abs()
    top = torch.finfo(torch.float16).max        # (of the key of weight 1 the sum passes it, and is infinite)
    check("dv", got["dv"][:, 0].clamp(-top, top), (val.clamp(-top, top), size + u * val.abs() + 2.0 ** -25))
    # where dq is not asked for, the same bits
    k1, v1 = (x.cuda().requires_grad_() for x in (k, v))
    out = lib.attend_prompt(q.cuda(), k1, v1, cu.cuda(), ck.cuda(), scale=1.0)
    dk, dv = torch.autograd.grad(out, (k1, v1), dout.cuda())
    assert torch.equal(dk, got["dk"]) and torch.equal(dv, got["dv"])


def test_views_of_negated_values(lib):
    """A tensor whose negation waits for its first use: taken as what it stands for, or refused."""
    import torch
    q, k, v, dout = [x.cuda() for x in make(5, [50], [50], 4, 2, 64, torch.bfloat16)]
    cu = lens_to_cu([50]).cuda()
    neg = torch._neg_view
    leaves = [neg(x).detach().requires_grad_() for x in (q, k, v)]
    out = lib.attend_prompt(*leaves, cu)
    got = (out,) + torch.autograd.grad(out, leaves, neg(dout))
    plain = [(-x).requires_grad_() for x in (q, k, v)]
    out = lib.attend_prompt(*plain, cu)
    want = (out,) + torch.autograd.grad(out, plain, -dout)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    cache = [torch.zeros(4, 2, 16, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    scale = torch.ones(4, 2, device="cuda")
    table, n = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.full((1,), 50, dtype=torch.int32, device="cuda")
    for c, x in (((*cache, neg(scale), scale), q), ((*cache, scale, scale), neg(q))):
        with pytest.raises(ValueError, match="negated"):
            lib.attend(x, c, table, cu, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [1, 4096])                 # keys in parts, each with its own largest weight, or whole
@pytest.mark.parametrize("n,m", [(1, 40000), (70, 20000), (300, 9000)])
def test_many_small_weights_in_fp16(lib, n, m, heads, D):
    """Weights of 2^-30 to 2^-24.5 of the largest, whose own value is 0: what they sum to.

    The bound of prompt_ref for out, with 2^-32 of the row's largest weight in place of 2^-25 (half a step of fp16
    below 2^-14 for weights held 2^7 times their size) and half a step of the result below 2^-14:
      u |out| + (u + 2 E + m 2^-23) sum_s P_s |v_s| + 2^-32 m max|v| + 2^-25."""
    import torch
    u = 2.0 ** -11
    g = torch.Generator().manual_seed(m + D)
    q, k = torch.zeros(n, 1, D, dtype=torch.float16), torch.zeros(m, 1, D, dtype=torch.float16)
    q[:, :, 0] = 1
    k[1:, 0, 0] = (-17.0 - 3.5 * torch.rand(m - 1, generator=g)).half()
    v = (1 + 0.25 * torch.randn(m, 1, D, generator=g)).half()
    v[0] = 0
    dev = [t.cuda().expand(-1, heads, -1) for t in (q, k, v)]
    out = lib.attend_prompt(*dev, lens_to_cu([n]).cuda(), lens_to_cu([m]).cuda(), scale=1.0)
    assert bool((out == out[:, :1]).all())
    x = k[:, 0, 0].double().expand(n, m).masked_fill(torch.arange(m) > m - n + torch.arange(n)[:, None], -torch.inf)
    P = torch.softmax(x, -1)
    assert float(P[:, 1:].max()) < 2.0 ** -24
    E = (D + 8) * 2.0 ** -24 * (2 * 20.5 + 0.1) + 2.0 ** -22
    val, size = P @ v[:, 0].double(), P @ v[:, 0].double().abs()
    tol = u * val.abs() + (u + 2 * E + m * 2.0 ** -23) * size + 2.0 ** -32 * m * float(v.abs().max()) + 2.0 ** -25
    assert float((tol / val).max()) < 0.25               # (so that sums without them are told apart)
    check("out", out[:, 0], (val, tol))
