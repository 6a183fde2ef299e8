"""Positions next to 2^31: a sequence whose last pages are all that is left of
it, at the end of the longest table that a call takes."""
import pytest

from tests.attend_ref import make_cache, ref_append, ref_attend, ref_packed
from tests.gpu_util import say
from tests.test_gpu_attend import _dev, _gen, _within

pytestmark = pytest.mark.gpu


def _end_of_a_table(page, T, D, seed):
    """The last `keep` pages of a table of 2^31 - 128 positions, and the same pages as a short sequence."""
    import torch
    g = _gen(seed)
    most, keep = (2 ** 31 - 128) // page, -(-640 // page)
    short = torch.randperm(keep, generator=g).int()[None]
    cache = make_cache(g, keep, 2, page, D)
    table = torch.full((1, most), -1, dtype=torch.int32, device="cuda")
    table[0, -keep:] = short[0].cuda()
    q = torch.randn(T, 8, D, generator=g).bfloat16()
    cu = torch.tensor([0, T]).int()
    return cache, table, most * page, short, keep * page, cu, q


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("T,D", [(1, 64), (9, 128), (80, 64)])
@pytest.mark.parametrize("window", [0, 300])
def test_attend_at_the_end_of_the_longest_table(lib, page, T, D, window):
    import torch
    cache, table, L, short, Ls, cu, q = _end_of_a_table(page, T, D, 95)
    say("far", page, T, D, window)
    out = lib.attend(q.cuda(), _dev(*cache), table, cu.cuda(), torch.tensor([L]).int().cuda(), window=window)
    ref, tol, _ = ref_attend(q, cache, short, cu, torch.tensor([Ls]).int(), D ** -0.5, window)
    _within(out, ref, tol, "far")


@pytest.mark.parametrize("page", [16, 128])
def test_lists_and_append_at_the_end_of_the_longest_table(lib, page):
    import torch
    T, D = 24, 64
    cache, table, L, short, Ls, cu, q = _end_of_a_table(page, T, D, 96)
    g = _gen(97)
    kl, kls, far = torch.tensor([L]).int().cuda(), torch.tensor([Ls]).int(), L - Ls
    idx = torch.stack([torch.randperm(Ls, generator=g)[:200] for _ in range(T)]).int()
    dc = _dev(*cache)
    say("far lists", page)
    out = lib.attend_selected(q.cuda(), dc, table, cu.cuda(), kl, (idx.long() + far).int().cuda())
    ref, tol, _ = ref_attend(q, cache, short, cu, kls, D ** -0.5, idx=idx)
    _within(out, ref, tol, "selected")
    shared = torch.stack([torch.randperm(Ls, generator=g) for _ in range(3)]).int()
    masks = torch.randint(0, 256, shared.shape, generator=g).int().view(torch.uint32)
    lens = torch.tensor([Ls, Ls, 99]).int()
    for group in (8, 24):    # few and many (row, head) pairs
        n = -(-T // group)
        out = lib.attend_packed(q.cuda(), dc, table, kl, *_dev((shared[:n].long() + far).int(), masks[:n].contiguous(), lens[:n]), group)
        ref, tol = ref_packed(q, cache, short, kls, shared[:n], masks[:n], lens[:n], group, D ** -0.5)
        _within(out, ref, tol, f"packed in {group}")
    k = torch.randn(T, 2, D, generator=g).bfloat16()
    want = ref_append(k, k, cache, short, cu, kls, None, False)
    lib.kv_append(*_dev(k, k), dc, table, cu.cuda(), kl)
    for a, b in zip(dc, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
