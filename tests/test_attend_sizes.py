"""Sizes at the ends of their ranges, without a GPU: what the kernels could not
number is refused as an argument error, before any device call."""
import pytest

import indexer_topk_long_amd as ltk
from tests.test_attend_abi import EINVAL, _append, _attend


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
