"""Rows of the paged cache read back, against the bytes' values."""
import pytest

from tests.attend_ref import dense_kv, make_batch, make_cache

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    return torch.Generator().manual_seed(seed)


def _want(cache, table, cu, kv_len, T, dtype):
    """k, v [T, Hkv, D] and written [T]: fp32 product rounded to dtype."""
    import torch
    page = cache[0].shape[2]
    k, v = (torch.zeros(T, cache[0].shape[1], cache[0].shape[3], dtype=dtype) for _ in range(2))
    written = torch.zeros(T, dtype=torch.bool)
    for b in range(table.shape[0]):
        r0, r1, n = int(cu[b]), int(cu[b + 1]), max(int(kv_len[b]), 0)
        kk, vv, _ = dense_kv(cache, table[b], n, page)     # zeros where there is no page
        for r in range(r0, r1):
            pos = n - (r1 - r0) + r - r0
            written[r] = True
            if pos >= 0:
                k[r], v[r] = kk[:, pos].float().to(dtype), vv[:, pos].float().to(dtype)
    return k, v, written


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_read(lib, page, D, dtype):
    import torch
    dt = getattr(torch, dtype)
    g = _gen(page + D)
    rows, lens = [1, 0, 130, 33, 5], [1, 40, 130, 300, 2]       # the last has rows before its first token
    table, cu, n, pages = make_batch(g, rows, lens, page)
    cache = make_cache(g, pages, 3, page, D, pow2=dtype != "float32")
    T = sum(rows) + 4                                            # rows behind the last sequence
    out = [torch.full((T, 3, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    c = [x.cuda() for x in cache]
    res = lib.kv_read(c, table.cuda(), cu.cuda(), n.cuda(), T, dtype=dt, out=tuple(out))
    assert res[0] is out[0] and res[1] is out[1]
    k, v, written = _want(cache, table, cu, n, T, dt)
    for got, want in zip(out, (k, v)):
        got = got.cpu()
        assert torch.equal(got[written], want[written]) and bool((got[~written] == 7).all())
    own = lib.kv_read(c, table.cuda(), cu.cuda(), n.cuda(), T, dtype=dt)
    assert all(torch.equal(a.cpu()[written], b[written]) and a.dtype == dt for a, b in zip(own, (k, v)))


def test_every_byte(lib):
    """All 256 bytes, NaN and negative zero among them, under scales at the range's ends."""
    import torch
    byte = torch.arange(256, dtype=torch.uint8).view(1, 1, 4, 64).repeat(3, 1, 4, 1)
    byte = byte.view(3, 1, 16, 64).contiguous()
    sc = torch.tensor([[2.0 ** -64], [1.0], [2.0 ** 64]])
    cache = (byte.view(torch.float8_e4m3fn), byte.view(torch.float8_e4m3fn), sc, sc)
    table, cu, n = (torch.tensor(x, dtype=torch.int32) for x in ([[0, 1, 2]], [0, 48], [48]))
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        k, v = lib.kv_read([x.cuda() for x in cache], table.cuda(), cu.cuda(), n.cuda(), 48, dtype=dt)
        want = (byte.view(torch.float8_e4m3fn).float() * sc[:, :, None, None]).transpose(1, 2).reshape(48, 1, 64).to(dt)
        for got in (k, v):
            got = got.cpu()
            assert torch.equal(got.isnan(), want.isnan())
            assert torch.equal(got.nan_to_num(nan=0.5), want.nan_to_num(nan=0.5))
            assert torch.equal(torch.signbit(got[~got.isnan()]), torch.signbit(want[~want.isnan()]))


def test_bad_pages_and_positions(lib):
    import torch
    g = _gen(5)
    table, cu, n, pages = make_batch(g, [90], [200], 16, max_pages=10)      # positions past the table
    table[0, 8] = -1
    table[0, 7] = pages
    cache = make_cache(g, pages, 2, 16, 64)
    k, v, written = _want(cache, table, cu, n, 90, torch.bfloat16)
    got = lib.kv_read([x.cuda() for x in cache], table.cuda(), cu.cuda(), n.cuda(), 90)
    assert torch.equal(got[0].cpu(), k) and torch.equal(got[1].cpu(), v)
    assert bool((k[-40:] == 0).all())


def test_what_append_wrote_comes_back(lib):
    """append, then read: within the rounding to e4m3 (half a step: 2^-4 of a value, 2^-10 of the scale for subnormals)."""
    import torch
    g = _gen(9)
    rows, lens = [40, 3], [57, 3]
    table, cu, n, pages = make_batch(g, rows, lens, 16)
    cache = [x.cuda() for x in make_cache(g, pages, 2, 16, 64)]
    k, v = (torch.randn(43, 2, 64, generator=g).bfloat16().cuda() for _ in range(2))
    lib.kv_append(k, v, cache, table.cuda(), cu.cuda(), n.cuda())
    got = lib.kv_read(cache, table.cuda(), cu.cuda(), n.cuda(), 43, dtype=torch.float32)
    for x, y, sc in zip((k, v), got, cache[2:]):
        assert bool(((x.float() - y).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -10 * float(sc.max())).all())


def test_a_prompt_read_back_is_attended_like_the_cache(lib):
    """kv_read, then attend_prompt over the rows: attend's result within both tolerances."""
    import torch
    from tests.attend_ref import ref_attend
    g = _gen(12)
    rows, lens = [9, 30], [120, 64]
    table, cu, n, pages = make_batch(g, rows, lens, 32)
    cache = make_cache(g, pages, 2, 32, 64)
    c = [x.cuda() for x in cache]
    q = torch.randn(39, 8, 64, generator=g).bfloat16()
    ck = torch.tensor([0, 120, 184], dtype=torch.int32).cuda()
    k, v = lib.kv_read(c, table.cuda(), ck, n.cuda(), 184)
    out = lib.attend_prompt(q.cuda(), k, v, cu.cuda(), ck)
    want, tol, _ = ref_attend(q, cache, table, cu, n, 0.125)
    # (weights in bf16, 2^-8 of themselves, where the cache's kernels round to fp16)
    extra = 2.0 ** -8 * float(v.abs().max())
    assert bool(((out.cpu().double() - want).abs() <= tol + extra).all())
    assert bool(((lib.attend(q.cuda(), c, table.cuda(), cu.cuda(), n.cuda()).cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("what", ["dtype", "T", "out shape", "out type", "out pair", "grad"])
def test_refusals(lib, what):
    import torch
    g = _gen(1)
    table, cu, n, pages = make_batch(g, [4], [4], 16)
    c = [x.cuda() for x in make_cache(g, pages, 2, 16, 64)]
    a = dict(T=4, dtype=torch.bfloat16, out=None)
    err = ValueError
    if what == "dtype":
        a["dtype"], err = torch.float64, TypeError
    elif what == "T":
        a["T"] = -1
    elif what == "out shape":
        a["out"] = (torch.empty(4, 2, 64, device="cuda").bfloat16(), torch.empty(3, 2, 64, device="cuda").bfloat16())
    elif what == "out type":
        a["out"], err = (torch.empty(4, 2, 64, device="cuda"),) * 2, TypeError
    elif what == "out pair":
        a["out"], err = torch.empty(4, 2, 64, device="cuda").bfloat16(), TypeError
    else:
        c[2].requires_grad_()
        err = RuntimeError
    with pytest.raises(err):
        lib.kv_read(c, table.cuda(), cu.cuda(), n.cuda(), **a)


def test_offsets_past_32_bits(lib):
    """Rows of outputs of more than 2^31 elements, from a cache of more than 2^31 bytes."""
    import torch
    Hkv, page, D, n = 128, 128, 128, 1100
    T = n * page
    ids = torch.randperm(n, generator=_gen(3)).int().cuda()
    byte = torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device="cuda")
    mark = (torch.arange(n * page, device="cuda") % 100 + 1).to(torch.uint8)
    byte.view(n, Hkv, page, D)[:, :, :, 0] = mark.view(n, 1, page)
    byte[:, :, :, D - 1] = torch.arange(Hkv, device="cuda").to(torch.uint8)[None, :, None]
    scale = torch.ones(n, Hkv, device="cuda")
    data = byte.view(torch.float8_e4m3fn)
    cu, kv_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [T]))
    k, v = lib.kv_read((data, data, scale, scale), ids[None], cu, kv_len, T)
    assert k.numel() > 1 << 31
    value = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).to(torch.bfloat16)
    want0 = value[mark.view(n, page)[ids.long()].reshape(-1).long()]
    for x in (k, v):
        assert torch.equal(x[:, 0, 0], want0) and torch.equal(x[:, Hkv - 1, 0], want0)
        # (byte 127 is NaN, whose sign is no matter)
        assert torch.equal(x[T - 1, :, D - 1].nan_to_num(nan=-1.0), value[:Hkv].nan_to_num(nan=-1.0))
        assert not bool(x[:, :, 1:D - 1].any())
