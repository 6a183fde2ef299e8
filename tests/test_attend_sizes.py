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
