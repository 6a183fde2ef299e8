"""Sizes at the ends of their ranges, without a GPU: what the kernels could not
number is refused as an argument error, before any device call."""
import pytest

import indexer_topk_long_amd as ltk
from tests.test_attend_abi import EINVAL, EWS, _append, _attend


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["append", "attend", "selected", "packed"])
def test_tables_whose_last_tile_passes_32_bits(kind, page):
    """max_pages * page_size <= 2^31 - 128: the end of a tile that begins in the table is an int32."""
    most = (2 ** 31 - 128) // page
    n_seq = dict(n_seq=1) if kind == "packed" else {}
    call = _append if kind == "append" else lambda **kw: _attend(kind, **kw)
    assert call(page_size=page, max_pages=most + 1, n_pages=4, **n_seq) == EINVAL
    assert call(page_size=page, max_pages=most, n_pages=4, T=0, **n_seq) == 0
    with pytest.raises(ltk.LtkError):
        ltk.attend_workspace_bytes(0, 4, 8, 4, 128, 1, (most + 1) * page)
    assert ltk.attend_workspace_bytes(0, 4, 8, 4, 128, 1, most * page) >= 256


MOST = 2 ** 31 - 256      # rows times query heads


@pytest.mark.parametrize("kind", ["append", "attend", "selected", "packed"])
@pytest.mark.parametrize("T,Hq", [(MOST + 1, 1), (1, MOST + 1), (MOST // 8 + 1, 8)])
def test_rows_times_heads_past_32_bits(kind, T, Hq):
    n_seq = dict(n_seq=1) if kind == "packed" else {}
    call = _append if kind == "append" else lambda **kw: _attend(kind, **kw)
    assert call(T=T, Hq=Hq, n_kv_heads=1, **n_seq) == EINVAL
    if kind != "append":
        with pytest.raises(ltk.LtkError):
            ltk.attend_workspace_bytes(["attend", "selected", "packed"].index(kind), T, Hq, 1, 128, 1, 64, 1)


@pytest.mark.parametrize("kind,group", [(0, 0), (1, 0), (2, 1), (2, 32)])
@pytest.mark.parametrize("T,Hq,Hkv", [(MOST, 1, 1), (MOST - 31, 1, 1), (1 << 20, 1 << 10, 1 << 10), (1 << 10, 1 << 20, 1)])
def test_workspaces_of_the_largest_calls(kind, group, T, Hq, Hkv):
    """Sizes whose sums pass 32 bits on the way: a refusal or a size that can be one (a few thousand parts of at most 256
    rows of 130 floats, and what the join reads)."""
    if kind == 2 and group * (Hq // Hkv) > 1 << 30:
        return
    try:
        n = ltk.attend_workspace_bytes(kind, T, Hq, Hkv, 128, 1, 2048, group)
    except ltk.LtkError:
        return
    assert 256 <= n <= 2048 * 256 * 130 * 4


@pytest.mark.parametrize("kw", [
    dict(n_seq=1 << 30),                                       # pages that can receive rows: 2 n_seq + ..
    dict(n_seq=1 << 21, n_kv_heads=8, Hq=8),                   # .. times heads, keys and values: 2^25 workgroups of 256
    dict(T=1 << 28, Hq=4, n_kv_heads=4, page_size=16),         # 2^24 pages
    dict(T=1 << 24, Hq=64, n_kv_heads=4, rot=2, n_seq=1),      # queries in single elements: 2^24 workgroups of 1,024
])
def test_appends_of_more_workgroups_than_a_launch_has(kw):
    assert _append(n_pages=4, **kw) == EINVAL


@pytest.mark.parametrize("kind,few,many", [
    ("selected", dict(T=(1 << 21) - 1, Hq=8, n_kv_heads=8), dict(T=1 << 21, Hq=8, n_kv_heads=8)),
    ("selected", dict(T=(1 << 20) - 1, Hq=64, n_kv_heads=1), dict(T=1 << 23, Hq=64, n_kv_heads=1)),
    ("packed", dict(T=(1 << 24) - 1, Hq=1, n_kv_heads=1, group=1, n_seq=1), dict(T=1 << 24, Hq=1, n_kv_heads=1, group=1, n_seq=1)),
])
def test_lists_of_more_workgroups_than_a_launch_has(kind, few, many):
    """Refused as an argument error; the next smaller call gets as far as its (too small) workspace."""
    assert _attend(kind, wsb=0, **few) == EWS
    assert _attend(kind, wsb=0, **many) == EINVAL
    kw = dict(group=0, **many) if kind == "selected" else many
    with pytest.raises(ltk.LtkError):
        ltk.attend_workspace_bytes(1 if kind == "selected" else 2, kw["T"], kw["Hq"], kw["n_kv_heads"], 128, 1, 64, kw["group"])


def test_a_cache_that_autograd_follows_is_refused():
    import torch
    i32 = torch.int32
    k = torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn)
    s = torch.ones(4, 2)
    batch = torch.zeros(1, 4, dtype=i32), torch.tensor([0, 1], dtype=i32), torch.ones(1, dtype=i32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    followed = k.clone().requires_grad_()
    with pytest.raises(RuntimeError, match="cache k requires grad"):
        ltk.attend(q, (followed, k, s, s), *batch)
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):     # the next check
        ltk.attend(q, (followed, k, s, s), *batch)


def _sizes(r):
    Hkv = r.choice([1, 2, 4, 8])
    Hq = Hkv * r.choice([1, 2, 4, 5, 8, 16, 40])
    kind = r.randint(0, 2)
    group = r.choice([1, 2, 8, 16, 32]) if kind == 2 else 0
    n_seq = 1 if kind == 2 else r.choice([1, 2, 7, 64, 300])
    log = lambda hi: int(round(2 ** r.uniform(0, hi)))
    return kind, log(13), Hq, Hkv, r.choice([64, 128]), n_seq, log(16 if kind else 20), group


def test_workspace_suffices_for_all_smaller_calls():
    """One buffer sized for the largest call serves calls of fewer rows, sequences and entries."""
    import random
    r = random.Random(1)
    for _ in range(3000):
        kind, T, Hq, Hkv, D, n, e, group = _sizes(r)
        size = ltk.attend_workspace_bytes(kind, T, Hq, Hkv, D, n, e, group)
        for _ in range(6):
            t, m, x = r.randint(1, T), r.randint(1, n), r.randint(1, e)
            if r.random() < 0.3:
                t = min(T, r.randint(1, 64))
            assert ltk.attend_workspace_bytes(kind, t, Hq, Hkv, D, m, x, group) <= size, (kind, T, t, Hq, Hkv, D, n, m, e, x, group)


def test_a_call_takes_what_the_size_function_gives():
    """Also where a smaller call sets the size; without a device the call ends after its checks."""
    import random
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    r = random.Random(2)
    for _ in range(1000):
        kind, T, Hq, Hkv, D, n, e, group = _sizes(r)
        page = 16
        e = -(-e // page) * page if kind == 0 else e
        size = ltk.attend_workspace_bytes(kind, T, Hq, Hkv, D, n, e, group)
        kw = dict(T=T, Hq=Hq, n_kv_heads=Hkv, head_dim=D, n_seq=n, page_size=page, wsb=size)
        kw.update({0: dict(max_pages=e // page), 1: dict(topk=e), 2: dict(cap=e, group=group)}[kind])
        rc = _attend(["attend", "selected", "packed"][kind], **kw)
        assert rc not in (EINVAL, EWS), kw


def test_workspace_of_a_long_packed_call_serves_its_first_groups():
    """64 heads on 8, groups of 16, lists of up to 32,768: 2,048 rows leave no list cut, 64 rows cut theirs."""
    size = lambda T: ltk.attend_workspace_bytes(2, T, 64, 8, 128, 1, 32768, 16)
    assert size(2048) >= size(512) >= size(64) > 1 << 24


@pytest.mark.parametrize("T,G", [(1, 1), (1 << 10, 1), (1 << 9, 64)])
def test_workspace_of_many_sequences_heads_and_positions(T, G):
    """Units times key tiles pass 64 bits where the batch has 2^31 sequences: the launch is the largest one there too."""
    size = lambda n, h: ltk.attend_workspace_bytes(0, T, h * G, h, 128, n, 2 ** 31 - 128)
    for h in (1, 64, 1 << 15):
        assert size(2 ** 31 - 1, h) == size(1 << 20, h) >= size(1 << 10, h)
