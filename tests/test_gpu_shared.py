"""Attention over shared first tokens against 64 bits and against attend."""
import pytest

from tests.attend_ref import make_cache, ref_attend

pytestmark = pytest.mark.gpu


def _gen(seed):
    import torch
    return torch.Generator().manual_seed(seed)


def shared_case(seed, groups, Hkv, G, page, D, own_pages=True, pow2=True, spread=1.0):
    """groups: list of (shared tokens or None, [(rows, tokens), ..]).  A group's sequences hold the ids of
    its shared pages; the page that its shared tokens end in is copied (own_pages) for each."""
    import torch
    g = _gen(seed)
    seqs = [x for _, ss in groups for x in ss]
    need = [-(-t // page) for _, t in seqs]
    pool = sum(need) + 4
    cache = make_cache(g, pool, Hkv, page, D, pow2, spread)
    ids = iter(torch.randperm(pool, generator=g).tolist())
    table = torch.full((len(seqs), max(need + [1])), -1, dtype=torch.int32)
    b, bounds, lens = 0, [0], []
    for shared, ss in groups:
        whole = (shared or 0) // page
        first = [next(ids) for _ in range(whole)]
        b0 = b
        for _, t in ss:
            n = -(-t // page)
            table[b, :whole] = torch.tensor(first, dtype=torch.int32)
            for p in range(whole, n):
                table[b, p] = next(ids)
            if shared and shared % page and b > b0:
                src, dst, off = int(table[b0, whole]), int(table[b, whole]), shared % page
                for x in cache[:2]:
                    x.view(torch.uint8)[dst, :, :off] = x.view(torch.uint8)[src, :, :off]
                for x in cache[2:]:
                    x[dst] = x[src]
            b += 1
        bounds.append(b)
        lens.append(shared or 0)
    cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).int()
    kv_len = torch.tensor([t for _, t in seqs], dtype=torch.int32)
    q = torch.randn(int(cu[-1]), Hkv * G, D, generator=g).bfloat16()
    return q, cache, table, cu, kv_len, torch.tensor(bounds, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)


def _check(lib, case, scale=None):
    import torch
    q, cache, table, cu, kv_len, bounds, lens = case
    d = [x.cuda() for x in cache]
    args = [x.cuda() for x in (table, cu, kv_len)]
    scale = scale or q.shape[2] ** -0.5
    want, tol, written = ref_attend(q, cache, table, cu, kv_len, scale)
    out = torch.full_like(q, 7.0).cuda()
    got = lib.attend_shared(q.cuda(), d, *args, bounds.cuda(), lens.cuda(), scale=scale, out=out)
    assert got is out
    got = got.cpu().double()
    assert bool(((got - want).abs() <= tol)[written].all()), float(((got - want).abs() - tol)[written].max())
    assert bool((got[~written] == 7).all())
    again = lib.attend_shared(q.cuda(), d, *args, bounds.cuda(), lens.cuda(), scale=scale)
    assert torch.equal(again.cpu()[written], got.bfloat16()[written])
    return got


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 16])
def test_decoding_answers(lib, G, D, page):
    seqs = lambda s, n: [(1, s + 1 + (17 * i) % 90) for i in range(n)]
    _check(lib, shared_case(page + D + G, [(300, seqs(300, 6)), (64, seqs(64, 2)), (17, seqs(17, 1))], 2, G, page, D))


@pytest.mark.parametrize("shared", [1, 15, 16, 31, 32, 33, 63, 64, 65, 500])
def test_borders(lib, shared):
    _check(lib, shared_case(shared, [(shared, [(1, shared + 1), (2, shared + 2), (3, shared + 60), (1, shared + 129)])],
                            1, 4, 16, 64))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared", [40, 4096])
def test_many_rows(lib, D, shared):
    """Groups and sequences of so many rows that the wide kernels take them."""
    _check(lib, shared_case(7, [(shared, [(20, shared + 30)] * 5 + [(90, shared + 200)])], 2, 8, 64, D))
    _check(lib, shared_case(8, [(shared, [(300, shared + 300), (150, shared + 400)]), (10, [(1, 90)])], 1, 8, 32, D))


def test_groups_that_share_nothing_and_sequences_in_none(lib):
    import torch
    case = list(shared_case(3, [(0, [(1, 40), (2, 90)]), (50, [(1, 70), (1, 51)]), (0, []), (20, [(1, 33)])], 2, 4, 16, 64))
    _check(lib, case)
    full = case[5].clone()
    case[5], case[6] = torch.tensor([2, 4], dtype=torch.int32), torch.tensor([50], dtype=torch.int32)
    _check(lib, case)                       # the sequences before and behind the group are on their own
    case[5], case[6] = torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    _check(lib, case)                       # no group at all
    case[5], case[6] = full, torch.zeros(4, dtype=torch.int32)
    _check(lib, case)


def test_sequences_without_rows_and_rows_behind(lib):
    import torch
    case = list(shared_case(4, [(60, [(0, 80), (1, 61), (0, 60), (2, 70)])], 2, 2, 16, 64))
    case[0] = torch.cat([case[0], torch.zeros(5, 4, 64, dtype=torch.bfloat16)])     # rows behind the last sequence
    _check(lib, case)
    case = shared_case(4, [(60, [(0, 80), (0, 61)])], 2, 2, 16, 64)
    _check(lib, case)


def test_value_scales_far_apart(lib):
    """Shared and own keys whose value scales are 2^100 apart, either way."""
    for hi, lo in ((2.0 ** 30, 2.0 ** -60), (2.0 ** -60, 2.0 ** 30)):
        q, cache, table, cu, kv_len, bounds, lens = shared_case(6, [(64, [(1, 100), (1, 90)])], 1, 4, 16, 64)
        cache[3][:] = lo
        cache[3][table[0, :4].long()] = hi
        _check(lib, (q, cache, table, cu, kv_len, bounds, lens))


def test_bytes_that_hold_no_key_may_be_anything(lib):
    import torch
    case = shared_case(9, [(40, [(1, 45), (3, 60)]), (90, [(1, 100)])], 2, 4, 32, 64)
    q, cache, table, cu, kv_len, bounds, lens = case
    used = torch.zeros(cache[0].shape[0], 32, dtype=torch.bool)
    for b in range(table.shape[0]):
        for p in range(-(-int(kv_len[b]) // 32)):
            n = min(32, int(kv_len[b]) - 32 * p)
            used[int(table[b, p]), :n] = True
    for x in cache[:2]:
        x.view(torch.uint8).permute(0, 2, 1, 3)[~used] = 0x7F
    for s in cache[2:]:
        s[~used.any(1)] = float("nan")
    _check(lib, case)


def test_pages_that_are_none(lib):
    import torch
    q, cache, table, cu, kv_len, bounds, lens = shared_case(10, [(64, [(1, 100), (2, 120)])], 2, 4, 16, 64)
    table[:, 1] = -1
    table[:, 2] = cache[0].shape[0]
    table[1, 6] = -5
    _check(lib, (q, cache, table, cu, kv_len, bounds, lens))
    table[:, :4] = -1                        # no shared key at all
    _check(lib, (q, cache, table, cu, kv_len, bounds, lens))
    table[:] = -1
    got = _check(lib, (q, cache, table, cu, kv_len, bounds, lens))
    assert bool((got == 0).all())


def test_lists_that_are_out_of_order(lib):
    """Nothing outside the tensors is touched, whatever groups and shared_len hold."""
    import torch
    q, cache, table, cu, kv_len, bounds, lens = shared_case(11, [(64, [(1, 100), (2, 120)]), (30, [(1, 40)])], 2, 4, 16, 64)
    d, args = [x.cuda() for x in cache], [x.cuda() for x in (table, cu, kv_len)]
    for g, s in (([5, -3, 2], [10, 10]), ([0, 100, -100], [2 ** 31 - 1, -5]), ([2, 2, 2], [64, 64]), ([0, 3, 1], [1000, 7])):
        lib.attend_shared(q.cuda(), d, *args, torch.tensor(g, dtype=torch.int32).cuda(), torch.tensor(s, dtype=torch.int32).cuda())
        torch.cuda.synchronize()


@pytest.mark.parametrize("D", [64, 128])
def test_long_prefix_cut_over_the_card(lib, D):
    """A prefix long enough to be cut into many parts: attend's result to within both roundings."""
    import torch
    S = 9000
    q, cache, table, cu, kv_len, bounds, lens = shared_case(12, [(S, [(1, S + 1 + 31 * i) for i in range(12)])], 2, 8, 64, D)
    d, args = [x.cuda() for x in cache], [x.cuda() for x in (table, cu, kv_len)]
    got = lib.attend_shared(q.cuda(), d, *args, bounds.cuda(), lens.cuda()).cpu()
    want, tol, _ = ref_attend(q[:3], cache, table[:3], cu[:4], kv_len[:3], D ** -0.5)
    assert bool(((got[:3].double() - want).abs() <= tol).all())
    plain = lib.attend(q.cuda(), d, *args).cpu().double()
    # both within the tolerance of the formula: its largest, for all rows alike
    assert bool(((got.double() - plain).abs() <= 2 * float(tol.max())).all())


def test_captured(lib):
    """Captured once, replayed while lengths, groups and queries change."""
    import torch
    a = shared_case(13, [(64, [(1, 100), (2, 120)]), (30, [(1, 40)])], 2, 4, 16, 64)
    q, cache, table, cu, kv_len, bounds, lens = [x.cuda() if hasattr(x, "cuda") else [y.cuda() for y in x] for x in a]
    ws = torch.empty(lib.attend_shared_workspace_bytes(4, 8, 2, 64, 3, 2, table.shape[1] * 16), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    call = lambda: lib.attend_shared(q, cache, table, cu, kv_len, bounds, lens, out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, (n, sl) in enumerate((([100, 120, 40], [64, 30]), ([90, 70, 33], [16, 3]), ([66, 120, 40], [0, 0]))):
        kv_len.copy_(torch.tensor(n)), lens.copy_(torch.tensor(sl))
        q.copy_(torch.randn(q.shape, generator=_gen(i)))
        graph.replay()
        torch.cuda.synchronize()
        held = out.clone()
        out.zero_()
        assert torch.equal(held, call())


def test_workspaces(lib):
    import torch
    q, cache, table, cu, kv_len, bounds, lens = shared_case(14, [(64, [(1, 100), (2, 120)])], 2, 4, 16, 64)
    d, args = [x.cuda() for x in cache], [x.cuda() for x in (table, cu, kv_len, bounds, lens)]
    need = lib.attend_shared_workspace_bytes(3, 8, 2, 64, 2, 1, table.shape[1] * 16)
    want = lib.attend_shared(q.cuda(), d, *args)
    guard = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = lib.attend_shared(q.cuda(), d, *args, workspace=guard[:need])
    assert torch.equal(got, want) and bool((guard[need:] == 0xA5).all())
    with pytest.raises(ValueError, match="workspace too small"):
        lib.attend_shared(q.cuda(), d, *args, workspace=guard[:1024])


@pytest.mark.parametrize("what,err", [("groups type", TypeError), ("groups size", ValueError), ("lens shape", ValueError),
                                      ("lens type", TypeError), ("cpu", ValueError), ("grad", RuntimeError)])
def test_refusals(lib, what, err):
    import torch
    q, cache, table, cu, kv_len, bounds, lens = [
        x.cuda() if hasattr(x, "cuda") else [y.cuda() for y in x]
        for x in shared_case(15, [(64, [(1, 100), (2, 120)])], 2, 4, 16, 64)]
    if what == "groups type":
        bounds = bounds.long()
    elif what == "groups size":
        bounds = torch.cat([bounds, bounds])
    elif what == "lens shape":
        lens = lens[None]
    elif what == "lens type":
        lens = lens.float()
    elif what == "cpu":
        bounds = bounds.cpu()
    else:
        q.requires_grad_()
    with pytest.raises(err):
        lib.attend_shared(q, cache, table, cu, kv_len, bounds, lens)


def test_many_groups(lib):
    """More groups and sequences than a workgroup looks at together."""
    groups = [(1 + (5 * i) % 40, [(1, 45 + i % 30)] * (1 + i % 2)) for i in range(290)]
    _check(lib, shared_case(16, groups, 1, 2, 16, 64))
