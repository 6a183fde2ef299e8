"""The paged e4m3 cache on the GPU: appended bytes and scales equal to the
plain fp64 form's, attention rows within the tolerance that attend_ref.py
derives, at the sizes and masks where a kernel can go wrong."""
import pytest

from tests.attend_ref import (make_batch, make_cache, poison, ref_append, ref_attend, ref_packed, rotate)
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    return torch.Generator().manual_seed(seed)


def _dev(*ts):
    return tuple(t if t is None else t.cuda() for t in ts)


def _within(got, ref, tol, what):
    import torch
    got = got.cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - ref).abs() > tol
    worst = ((got - ref).abs() / tol.clamp(min=1e-30)).max().item() if got.numel() else 0.0
    say(f"  {what}: worst error {worst:.3f} of the tolerance")
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.2f}"


# --------------------------------------------------------------- append

APPEND = [
    # rows per sequence, lengths, Hkv, Hq, page, D, rot, interleaved
    ([1], [1], 1, 1, 16, 64, 64, False),                       # the first token
    ([1], [1000000], 2, 6, 64, 128, 128, False),               # a far position in a page begun before
    ([1, 1, 1], [16, 17, 33], 2, 4, 16, 64, 64, True),         # slot 15, slot 0, slot 0
    ([5, 0, 3, 40], [5, 9, 100, 75], 4, 4, 32, 128, 64, False),  # an empty sequence; pages begun and ended inside
    ([70], [70], 3, 21, 16, 128, 24, True),                    # many small pages, rot in vectors of 4
    ([131], [190], 2, 2, 128, 64, 6, False),                   # rot in single elements
    ([300], [777], 1, 8, 64, 128, 0, False),                   # no rotation
    ([33, 33], [33, 50], 2, 2, 64, 128, 126, True),
    ([7], [3], 2, 4, 16, 64, 64, False),                       # more rows than tokens: the first have no position
    ([129], [129], 1, 1, 128, 128, 10, False),                 # widest page in single elements
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{c[0]}_{c[1]}_h{c[2]}_p{c[4]}_d{c[5]}_r{c[6]}{'i' if c[7] else ''}")
def test_append_vs_plain(lib, case):
    import torch
    rows, lens, Hkv, Hq, page, D, rot, il = case
    say("append", case)
    g = _gen(11)
    far = max(lens) > 100000
    if far:   # a sequence whose earlier pages are all one page: only its last page matters here
        table, cu, n = torch.zeros(1, -(-lens[0] // page), dtype=torch.int32), torch.tensor([0, 1]).int(), torch.tensor(lens).int()
        table[0, -1], pages = 2, 4
    else:
        table, cu, n, pages = make_batch(g, rows, lens, page)
    cache = make_cache(g, pages, Hkv, page, D)
    T = sum(rows)
    k = (torch.randn(T, Hkv, D, generator=g) * torch.exp2(2 * torch.randn(T, Hkv, 1, generator=g))).bfloat16()
    v = (torch.randn(T, Hkv, D, generator=g) * torch.exp2(2 * torch.randn(T, Hkv, 1, generator=g))).bfloat16()
    q = torch.randn(T, Hq, D, generator=g).bfloat16()
    f = None if rot == 0 else 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    want = ref_append(k, v, cache, table, cu, n, f, il)
    dc = _dev(*cache)
    qo = lib.kv_append(*_dev(k, v), dc, *_dev(table, cu, n, f, q), interleaved=il)
    for name, a, b in zip(("k", "v", "k_scale", "v_scale"), dc, want):
        a, b = a.cpu(), b
        if a.dtype == torch.float32:
            assert torch.equal(a, b), name
        else:
            d = a.view(torch.uint8) != b.view(torch.uint8)
            assert not d.any(), f"{name}: {int(d.sum())} bytes differ"
    # queries: half a bf16 step, and the fp32 rotation's three roundings on |a| + |b|
    pos = torch.cat([torch.arange(l - r, l) for r, l in zip(rows, lens)])
    ref = q.double() if f is None else rotate(q.double(), pos, f, il)
    tol = 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -24 * 2 * q.double().abs().amax(-1, keepdim=True)
    _within(qo, ref, tol, "queries")


def test_append_border_amax_zero_and_huge(lib):
    """Scales at their borders: amax exactly 448 s (1.75 x a power of two), just above it, zero rows, and magnitudes
    past 448 x 2^64, which saturate; a second call of the same rows changes nothing."""
    import torch
    page, D, Hkv = 16, 64, 6
    g = _gen(12)
    table, cu, n, pages = make_batch(g, [5], [5], page)
    cache = make_cache(g, pages, Hkv, page, D)
    v = torch.randn(5, Hkv, D, generator=g).bfloat16().clamp(-1, 1)
    v[2, 0, 3] = 1.75
    v[2, 1, 3] = 1.7578125            # the next bf16 above 1.75
    v[:, 2] = 0
    v[1, 3, 0] = 3e38
    v[:, 4] = v[:, 4] * 2.0 ** -90
    k = v.flip(1).contiguous()
    want = ref_append(k, v, cache, table, cu, n, None, False)
    dc = _dev(*cache)
    args = _dev(k, v), _dev(table, cu, n)
    for _ in range(2):
        assert lib.kv_append(*args[0], dc, *args[1]) is None
        for a, b in zip(dc, want):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    assert float(dc[3][table[0, 0].item(), 0]) == 2.0 ** -8 and float(dc[3][table[0, 0].item(), 1]) == 2.0 ** -7


def test_append_leaves_the_rest_alone(lib):
    """Rows before cu[0] and behind cu[B], bad page ids, tokens past the table, unused slots and pages."""
    import torch
    page, D, Hkv = 16, 128, 2
    g = _gen(13)
    table = torch.tensor([[3, -1, 1], [0, 4, 99], [2, 5, 6]], dtype=torch.int32)
    cu, n = torch.tensor([2, 42, 52, 72]).int(), torch.tensor([40, 48, 55]).int()   # the third ends past its table
    cache = make_cache(g, 8, Hkv, page, D)
    T = 75
    k = torch.randn(T, Hkv, D, generator=g).bfloat16()
    v, q = torch.randn(T, Hkv, D, generator=g).bfloat16(), torch.randn(T, 4, D, generator=g).bfloat16()
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    want = ref_append(k, v, cache, table, cu, n, f, False)
    dc = _dev(*cache)
    qo = torch.full((T, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.kv_append(*_dev(k, v), dc, *_dev(table, cu, n, f, q), q_out=qo)
    for a, b in zip(dc, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    assert bool((qo[:2] == 7).all()) and bool((qo[72:] == 7).all()) and not bool((qo[2:72] == 7).all(-1).any())


def test_append_token_by_token_equals_its_pages(lib):
    """One call per token: scales grow as the page fills, bytes are rounded again to them; queries rotated in place."""
    import torch
    page, D, Hkv, N = 16, 64, 2, 40
    g = _gen(14)
    table, cu, _, pages = make_batch(g, [1], [N], page)
    cache = make_cache(g, pages, Hkv, page, D)
    k = (torch.randn(N, Hkv, D, generator=g) * torch.exp2(torch.arange(N) * 0.3)[:, None, None]).bfloat16()
    v = (torch.randn(N, Hkv, D, generator=g) * torch.exp2(3 * torch.randn(N, Hkv, 1, generator=g))).bfloat16()
    f = 500.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    want, dc = cache, _dev(*cache)
    t, c, ff = _dev(table, cu, f)
    for i in range(N):
        n = torch.tensor([i + 1]).int()
        want = ref_append(k[i:i + 1], v[i:i + 1], want, table, cu, n, f, False)
        lib.kv_append(*_dev(k[i:i + 1], v[i:i + 1]), dc, t, c, n.cuda(), ff)
    for a, b in zip(dc, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


# --------------------------------------------------------------- attend

ATTEND = [
    # rows, lengths, Hkv, G, page, D, window, sinks
    ([1], [1], 1, 1, 16, 64, 0, 0),                            # one token
    ([1], [31], 2, 3, 16, 128, 0, 0),                          # pages end inside a tile
    ([1, 1, 1, 1], [32, 33, 1000, 4097], 2, 8, 64, 128, 0, 0),
    ([3, 0, 1, 8], [3, 12, 700, 260], 2, 4, 32, 64, 0, 0),     # an empty sequence, several rows
    ([5], [5], 1, 16, 16, 64, 0, 0),                           # a prompt from its first token
    ([1], [300], 1, 64, 128, 128, 0, 0),                       # one key/value head for 64
    ([2], [513], 3, 7, 16, 64, 0, 0),
    ([1], [2000], 2, 4, 64, 128, 100, 4),                      # window and sinks
    ([40], [400], 2, 2, 16, 64, 33, 5),
    ([9], [300], 1, 8, 32, 128, 1, 0),                         # a window of one: the row itself
    ([9], [300], 1, 8, 32, 128, 64, 64),
    ([70], [70], 2, 4, 64, 64, 16, 100),                       # more sinks than the window has left out
    ([1], [90], 2, 4, 16, 64, 1000, 4),                        # a window wider than the sequence
    ([130, 1, 257], [130, 500, 700], 2, 4, 64, 128, 0, 0),     # chunks
    ([200], [1500], 1, 5, 128, 64, 257, 3),
    ([6], [4], 2, 2, 16, 64, 0, 0),                            # more rows than tokens: the first see nothing
    ([2, 2], [0, 40], 2, 2, 16, 64, 0, 0),                     # a sequence of no tokens
]


def _attend_case(rows, lens, Hkv, G, page, D, seed, pow2=True, qscale=1.5):
    import torch
    g = _gen(seed)
    table, cu, n, pages = make_batch(g, rows, lens, page)
    cache = make_cache(g, pages, Hkv, page, D, pow2=pow2)
    poison(cache, table, lens, page)
    q = (qscale * torch.randn(sum(rows), Hkv * G, D, generator=g)).bfloat16()
    return cache, table, cu, n, q


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{c[0]}_{c[1]}_h{c[2]}x{c[3]}_p{c[4]}_d{c[5]}_w{c[6]}s{c[7]}")
def test_attend_vs_plain(lib, case):
    import torch
    rows, lens, Hkv, G, page, D, window, sinks = case
    say("attend", case)
    cache, table, cu, n, q = _attend_case(rows, lens, Hkv, G, page, D, 21)
    dc, db = _dev(*cache), _dev(table, cu, n)
    out = lib.attend(q.cuda(), dc, *db, window=window, n_sink=sinks)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, window, sinks)
    _within(out, ref, tol, "attend")
    again = lib.attend(q.cuda(), dc, *db, window=window, n_sink=sinks)
    assert torch.equal(out, again)


@pytest.mark.parametrize("pow2,qscale,scale", [(False, 1.5, None), (True, 40.0, None), (True, 1.0, -0.5), (False, 1.0, 0.0)])
def test_attend_scales(lib, pow2, qscale, scale):
    """Page scales that are no powers of two, sharp softmaxes, negative and zero score scales."""
    cache, table, cu, n, q = _attend_case([1, 20], [900, 300], 2, 4, 32, 128, 22, pow2, qscale)
    cache[3].mul_(2.0 ** 20), cache[2].mul_(2.0 ** -3)
    out = lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n), scale=scale)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 128 ** -0.5 if scale is None else scale)
    _within(out, ref, tol, f"pow2={pow2} q x {qscale} scale {scale}")


def test_attend_value_scales_far_apart(lib):
    """Value scales from 2^-60 to 2^60 across the pages of one sequence."""
    import torch
    cache, table, cu, n, q = _attend_case([1], [16 * 12], 1, 4, 16, 64, 23)
    cache[3][table[0].long()] *= torch.exp2(torch.linspace(-60, 60, 12).round())[:, None]
    out = lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n))
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 0.125)
    _within(out, ref, tol, "far apart")


def test_attend_freed_pages_and_rows_outside(lib):
    """Pages before a window given back (their ids gone, their bytes NaN), bad ids in the middle, tokens past the table,
    rows before cu[0] and behind cu[B] left as they were."""
    import torch
    page, D, Hkv, G = 16, 64, 2, 4
    g = _gen(24)
    table, cu, n, pages = make_batch(g, [2, 3, 4], [400, 200, 100], page)
    table[0, 1:20] = torch.tensor([-1, 10 ** 6, -2 ** 31] * 7)[:19].int()     # window 64, 4 sinks: pages 1..19 unseen
    table[1, 3] = pages                                                        # a hole
    cache = make_cache(g, pages, Hkv, page, D)
    poison(cache, table, [400, 200, 100], page)
    q = torch.randn(14, Hkv * G, D, generator=g).bfloat16()
    cu = cu + 2
    out = torch.full((14, Hkv * G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n), window=64, n_sink=4, out=out)
    ref, tol, written = ref_attend(q, cache, table, cu, n, D ** -0.5, 64, 4)
    assert bool((out.cpu()[~written] == 9).all()) and int(written.sum()) == 9
    _within(out.cpu()[written], ref[written], tol[written], "freed pages")
    short = table[:, :9].contiguous()                                          # 144 positions: the rest has no page
    out = lib.attend(q.cuda(), _dev(*cache), *_dev(short, cu, n))
    ref, tol, _ = ref_attend(q, cache, short, cu, n, D ** -0.5)
    _within(out.cpu()[written], ref[written], tol[written], "past the table")


def test_attend_random_batches(lib):
    """40 drawn batches of every head layout, page size and dimension."""
    import random
    r = random.Random(5)
    for i in range(40):
        B = r.randint(1, 5)
        rows = [r.choice([0, 1, 1, 2, r.randint(1, 50)]) for _ in range(B)]
        lens = [x + r.choice([0, r.randint(0, 40), r.randint(0, 600)]) for x in rows]
        Hkv, G, page, D = r.choice([1, 2, 3]), r.choice([1, 2, 3, 5, 8, 16, 17, 33]), r.choice([16, 32, 64, 128]), r.choice([64, 128])
        window, sinks = r.choice([(0, 0), (r.randint(1, 200), r.choice([0, 1, 30, 100]))])
        if sum(rows) == 0:
            continue
        say("batch", i, rows, lens, Hkv, G, page, D, window, sinks)
        cache, table, cu, n, q = _attend_case(rows, lens, Hkv, G, page, D, 100 + i)
        out = lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n), window=window, n_sink=sinks)
        ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, window, sinks)
        _within(out, ref, tol, "attend")


def test_attend_cache_past_4_gib(lib):
    """Pages whose byte offsets pass 2^32."""
    import torch
    page, D, Hkv = 128, 128, 8
    pages = (1 << 32) // (page * D * Hkv) + 40
    g = _gen(25)
    small = make_cache(g, 6, Hkv, page, D)
    table_s, cu, n, _ = make_batch(g, [2], [700], page, spare=0)
    k = torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros_like(k.view(torch.uint8)).view(torch.float8_e4m3fn)
    ks = torch.ones(pages, Hkv, device="cuda")
    vs = torch.ones(pages, Hkv, device="cuda")
    at = torch.tensor([pages - 1, 3, pages - 30, 1 << 12, pages // 2, pages - 2])
    for dst, src in zip((k, v), small[:2]):
        dst.view(torch.uint8)[at.cuda()] = src.view(torch.uint8).cuda()
    ks[at.cuda()], vs[at.cuda()] = small[2].cuda(), small[3].cuda()
    table = at[table_s.long()].int()
    q = torch.randn(2, 16, D, generator=g).bfloat16()
    ref, tol, _ = ref_attend(q, small, table_s, cu, n, D ** -0.5)
    out = lib.attend(q.cuda(), (k, v, ks, vs), *_dev(table, cu, n))
    _within(out, ref, tol, "dense")
    idx = torch.stack([torch.randperm(700, generator=g)[:300] for _ in range(2)]).int()
    ref, tol, _ = ref_attend(q, small, table_s, cu, n, D ** -0.5, idx=idx)
    _within(lib.attend_selected(q.cuda(), (k, v, ks, vs), *_dev(table, cu, n, idx)), ref, tol, "selected")
    nk = torch.randn(2, Hkv, D, generator=g).bfloat16()
    want = ref_append(nk, nk, small, table_s, cu, n, None, False)
    lib.kv_append(*_dev(nk, nk), (k, v, ks, vs), *_dev(table, cu, n))
    assert torch.equal(k.view(torch.uint8)[at.cuda()].cpu(), want[0].view(torch.uint8))
    assert torch.equal(vs[at.cuda()].cpu(), want[3])


# -------------------------------------------------------------- selected

SELECTED = [
    # rows, lengths, Hkv, G, page, D, topk
    ([1], [1], 1, 1, 16, 64, 1),
    ([1, 2], [500, 40], 2, 8, 64, 128, 31),
    ([3], [5000], 2, 4, 32, 128, 2049),                        # past one staged chunk
    ([2], [9000], 1, 64, 64, 64, 4500),
    ([1, 0, 5], [64, 3, 90], 3, 7, 16, 64, 128),               # longer lists than tokens: padded
    ([300], [700], 1, 2, 16, 64, 33),
    ([2], [300], 2, 17, 16, 128, 100),
]


def _lists(g, rows, lens, topk, junk=True):
    """Distinct positions up to each row's own, shuffled, -1 behind; some entries no keys."""
    import torch
    out = []
    for r, n in zip(rows, lens):
        for i in range(r):
            pos = n - r + i
            e = torch.full((topk,), -1, dtype=torch.int64)
            m = min(topk, pos + 1)
            e[:m] = torch.randperm(pos + 1, generator=g)[:m]
            if junk and topk > 8:
                e[1], e[3], e[5] = pos + 1, n + 1000, -7
            out.append(e[torch.randperm(topk, generator=g)])
    return torch.stack(out).int()


@pytest.mark.parametrize("case", SELECTED, ids=lambda c: f"{c[0]}_{c[1]}_h{c[2]}x{c[3]}_p{c[4]}_d{c[5]}_k{c[6]}")
def test_selected_vs_plain(lib, case):
    import torch
    rows, lens, Hkv, G, page, D, topk = case
    say("selected", case)
    cache, table, cu, n, q = _attend_case(rows, lens, Hkv, G, page, D, 31)
    idx = _lists(_gen(32), rows, lens, topk)
    args = (q.cuda(), _dev(*cache), *_dev(table, cu, n, idx))
    out = lib.attend_selected(*args)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, idx=idx)
    _within(out, ref, tol, "selected")
    assert torch.equal(out, lib.attend_selected(*args))


def test_selected_rows_without_keys(lib):
    import torch
    cache, table, cu, n, q = _attend_case([4], [100], 2, 4, 16, 64, 33)
    idx = torch.full((4, 50), -1, dtype=torch.int32)
    idx[1, 17] = 96          # the row itself is at 97
    idx[2, :] = 99           # after the row
    idx[3, 0], idx[3, 49] = 99, 2 ** 31 - 1
    out = torch.full_like(q, 5.0).cuda()
    lib.attend_selected(q.cuda(), _dev(*cache), *_dev(table, cu, n, idx), out=out)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 0.125, idx=idx)
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    _within(out, ref, tol, "sparse lists")


def test_selected_of_every_key_equals_attend(lib):
    """A list of all causal keys, repeated entries counted each time they appear."""
    import torch
    cache, table, cu, n, q = _attend_case([3], [200], 2, 4, 32, 128, 34)
    idx = torch.arange(200).repeat(3, 1).int()
    a = lib.attend_selected(q.cuda(), _dev(*cache), *_dev(table, cu, n, idx))
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 128 ** -0.5)
    _within(a, ref, tol, "all keys")
    idx[:, 150:] = 7
    a = lib.attend_selected(q.cuda(), _dev(*cache), *_dev(table, cu, n, idx))
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 128 ** -0.5, idx=idx)
    _within(a, ref, tol, "repeats")


# ---------------------------------------------------------------- packed

PACKED = [
    # T, length, Hkv, G, page, D, topk, group
    (1, 1, 1, 1, 16, 64, 1, 1),
    (37, 300, 2, 7, 16, 64, 60, 8),
    (64, 2000, 2, 8, 64, 128, 200, 16),
    (33, 500, 1, 4, 32, 128, 100, 32),
    (50, 50, 2, 2, 16, 64, 40, 5),
    (20, 6000, 1, 16, 128, 64, 1500, 16),
    (7, 400, 2, 40, 64, 128, 90, 3),
    (16, 900, 4, 1, 64, 64, 128, 16),
    (100, 1000, 1, 3, 16, 128, 64, 1),
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"T{c[0]}_L{c[1]}_h{c[2]}x{c[3]}_p{c[4]}_d{c[5]}_k{c[6]}_g{c[7]}")
def test_packed_vs_plain(lib, case):
    import torch
    T, L, Hkv, G, page, D, topk, group = case
    say("packed", case)
    cache, table, cu, n, q = _attend_case([T], [L], Hkv, G, page, D, 41)
    idx = _lists(_gen(42), [T], [L], topk)
    dc, dt, dn = _dev(*cache), table.cuda(), n.cuda()
    sh, m, ln = lib.dsa_pack(idx.cuda(), L, group)
    out = lib.attend_packed(q.cuda(), dc, dt, dn, sh, m, ln, group)
    ref, tol = ref_packed(q, cache, table, n, sh.cpu(), m.cpu(), ln.cpu(), group, D ** -0.5)
    _within(out, ref, tol, "packed")
    # the packed lists hold exactly each row's own selection
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, idx=idx)
    _within(out, ref, tol, "packed against the rows' own lists")
    assert torch.equal(out, lib.attend_packed(q.cuda(), dc, dt, dn, sh, m, ln, group))


def test_packed_odd_lists(lib):
    """Lengths past cap and below 0, bits of rows that are not there, keys after a row, entries that are no keys, a hole
    in the table, groups with nothing."""
    import torch
    T, L, group, cap = 21, 160, 8, 70
    cache, table, cu, n, q = _attend_case([T], [L], 2, 4, 16, 64, 43)
    table[0, 4] = -1
    poison(cache, table, [L], 16)
    g = _gen(44)
    shared = torch.stack([torch.randperm(L + 20, generator=g)[:cap] for _ in range(3)]).int()
    shared[:, 5], shared[1, 9] = -3, 2 ** 31 - 1
    masks = torch.randint(0, 2 ** 31 - 1, (3, cap), generator=g).int()
    masks[0] &= ~(1 << 2)            # row 2 selects nothing
    lens = torch.tensor([cap + 50, cap, -4]).int()
    out = lib.attend_packed(q.cuda(), _dev(*cache), *_dev(table, n, shared, masks.view(torch.uint32), lens), group)
    ref, tol = ref_packed(q, cache, table, n, shared, masks.view(torch.uint32), lens, group, 0.125)
    assert bool((out[2] == 0).all()) and bool((out[16:] == 0).all())
    _within(out, ref, tol, "odd lists")


# ----------------------------------------------------- together, and streams

def test_append_select_attend_together(lib):
    """A prompt and decode steps as they are run: append, select by the indexer, attend to the selection, packed and
    not, each step against the plain forms on the bytes that the cache holds."""
    import torch
    g = _gen(51)
    page, D, Hkv, Hq, N, topk, H = 32, 64, 2, 8, 300, 64, 4
    table, _, _, pages = make_batch(g, [N], [N + 40], page)
    zero = torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda")
    cache = (zero.view(torch.float8_e4m3fn), zero.clone().view(torch.float8_e4m3fn),
             torch.zeros(pages, Hkv, device="cuda"), torch.zeros(pages, Hkv, device="cuda"))
    host = tuple(t.cpu() for t in cache)
    f = 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    ik = torch.randn(N + 40, D, generator=g).bfloat16().cuda()
    dt = table.cuda()
    at = 0
    for rows in (N, 1, 1, 8, 1):
        n = at + rows
        k, v = (torch.randn(rows, Hkv, D, generator=g).bfloat16() for _ in range(2))
        q = torch.randn(rows, Hq, D, generator=g).bfloat16()
        cu, kl = torch.tensor([0, rows]).int(), torch.tensor([n]).int()
        host = ref_append(k, v, host, table, cu, kl, f, False)
        qr = lib.kv_append(*_dev(k, v), cache, dt, *_dev(cu, kl, f, q))
        for a, b in zip(cache, host):
            assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
        iq, w = torch.randn(rows, H, D, generator=g).bfloat16().cuda(), torch.rand(rows, H, generator=g).cuda()
        pos = torch.arange(at, n, dtype=torch.int32, device="cuda")
        idx = lib.score_select(iq, ik[:n], w, pos, topk)
        out = lib.attend_selected(qr, cache, dt, *_dev(cu, kl), idx)
        ref, tol, _ = ref_attend(qr.cpu(), host, table, cu, kl, D ** -0.5, idx=idx.cpu())
        _within(out, ref, tol, f"selected, {rows} rows")
        sh, m, ln = lib.dsa_pack(idx, n, 8)
        _within(lib.attend_packed(qr, cache, dt, kl.cuda(), sh, m, ln, 8), ref, tol, f"packed, {rows} rows")
        ref, tol, _ = ref_attend(qr.cpu(), host, table, cu, kl, D ** -0.5, window=50, n_sink=4)
        _within(lib.attend(qr, cache, dt, *_dev(cu, kl), window=50, n_sink=4), ref, tol, f"window, {rows} rows")
        at = n


def test_captured_and_replayed(lib):
    """The step captured once and replayed with new rows, lengths and lists in the same buffers, eager work between."""
    import torch
    page, D, Hkv, G, B, topk = 16, 64, 2, 4, 3, 40
    g = _gen(52)
    lens = [100, 33, 250]
    table, cu, n, pages = make_batch(g, [1] * B, [x + 8 for x in lens], page)
    cache = make_cache(g, pages, Hkv, page, D)
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    dc = _dev(*cache)
    dt, dcu, df = _dev(table, cu, f)
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(B, topk, dtype=torch.int32, device="cuda")

    def step():
        qr = lib.kv_append(k, v, dc, dt, dcu, kl, df, q=q)
        return lib.attend(qr, dc, dt, dcu, kl), lib.attend_selected(qr, dc, dt, dcu, kl, idx)

    eager = tuple(t.clone() for t in dc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(dc, eager):
        a.copy_(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(5):
        cur = [x + 1 + i for x in lens]
        kl.copy_(torch.tensor(cur).int())
        k.copy_(torch.randn(k.shape, generator=g)), v.copy_(torch.randn(k.shape, generator=g))
        q.copy_(torch.randn(q.shape, generator=g))
        idx.copy_(_lists(g, [1] * B, cur, topk))
        saved = tuple(t.clone() for t in dc)
        graph.replay()
        torch.cuda.synchronize()
        got, after = [o.clone() for o in outs], tuple(t.clone() for t in dc)
        for a, b in zip(dc, saved):
            a.copy_(b)
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {i}"
        for a, b in zip(after, dc):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}"


def test_two_streams_at_once(lib):
    """Calls on two streams with their own workspaces give what they give alone."""
    import torch
    cases = [_attend_case([1, 1], [5000, 300], 2, 8, 64, 128, 53), _attend_case([4], [3000], 2, 4, 32, 64, 54)]
    args = [(q.cuda(), _dev(*c), *_dev(t, cu, n)) for c, t, cu, n, q in cases]
    alone = [lib.attend(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = [[], []]
    for _ in range(5):
        for i, (s, a) in enumerate(zip(streams, args)):
            with torch.cuda.stream(s):
                got[i].append(lib.attend(*a))
    torch.cuda.synchronize()
    for g, w in zip(got, alone):
        assert all(torch.equal(x, w) for x in g)


def test_workspace_argument_and_refusals(lib):
    import torch
    import indexer_topk_long_amd as ltk
    cache, table, cu, n, q = _attend_case([1], [5000], 2, 8, 64, 128, 55)
    a = (q.cuda(), _dev(*cache), *_dev(table, cu, n))
    need = ltk.attend_workspace_bytes(0, 1, 16, 2, 128, 1, table.shape[1] * 64)
    ws = torch.full((need,), 0x7F, dtype=torch.uint8, device="cuda")   # a used workspace
    assert torch.equal(lib.attend(*a, workspace=ws), lib.attend(*a))
    with pytest.raises(ValueError, match="workspace too small"):
        lib.attend(*a, workspace=ws[:need - 1])
    with pytest.raises(TypeError):
        lib.attend(a[0].float(), *a[1:])
    with pytest.raises(ValueError, match="not a multiple"):
        lib.attend(a[0][:, :15].contiguous(), *a[1:])
    with pytest.raises(ValueError, match="contiguous"):
        lib.attend(torch.zeros(1, 16, 256, dtype=torch.bfloat16, device="cuda")[..., ::2], *a[1:])
    with pytest.raises(ValueError, match="cu must be"):
        lib.attend(*a[:3], a[3][:1], a[4])
    with pytest.raises(ltk.LtkError):
        lib.attend(*a, window=-1)
    with pytest.raises(ltk.LtkError):
        lib.attend(*a, scale=float("inf"))
    with pytest.raises(ValueError, match="q_out without q"):
        lib.kv_append(torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda"), *a[1:], q_out=a[0])
    empty = lib.attend(a[0][:0], a[1], a[2], torch.zeros_like(a[3]), a[4])
    assert empty.shape == (0, 16, 128)
