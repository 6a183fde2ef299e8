"""Reading the cache back where a call ends inside a sequence."""
import pytest

from tests.attend_ref import make_batch, make_cache
from tests.test_gpu_kv_read import _gen, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 40, 41, 60, 139, 140])
def test_fewer_rows_than_the_sequences_have(lib, T):
    """Row cu[b] + i is the token at kv_len[b] - (cu[b + 1] - cu[b]) + i, however many rows are asked for."""
    import torch
    g = _gen(31)
    rows, lens = [40, 0, 100], [55, 9, 100]
    table, cu, n, pages = make_batch(g, rows, lens, 16)
    cache = make_cache(g, pages, 2, 16, 64)
    k, v, _ = _want(cache, table, cu, n, 140, torch.bfloat16)
    got = lib.kv_read([x.cuda() for x in cache], table.cuda(), cu.cuda(), n.cuda(), T)
    assert torch.equal(got[0].cpu(), k[:T]) and torch.equal(got[1].cpu(), v[:T])


def test_offsets_at_the_ends_of_32_bits(lib):
    """Positions of offsets 2^32 apart: before every token, so zeros."""
    import torch
    g = _gen(32)
    table, cu, n, pages = make_batch(g, [20], [20], 16)
    cache = [x.cuda() for x in make_cache(g, pages, 2, 16, 64)]
    cu = torch.tensor([-(2 ** 31), 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for x in lib.kv_read(cache, table.cuda(), cu, n.cuda(), 20):
        assert not bool(x.any())


def test_out_tensors_that_share_memory_are_refused(lib):
    import torch
    g = _gen(33)
    table, cu, n, pages = make_batch(g, [20], [20], 16)
    cache = [x.cuda() for x in make_cache(g, pages, 2, 16, 64)]
    args = cache, table.cuda(), cu.cuda(), n.cuda(), 20
    both = torch.zeros(40, 2, 64, dtype=torch.bfloat16, device="cuda")
    for pair in ((both[:20],) * 2, (both[:20], both[19:39]), (both[1:21], both[:20])):
        with pytest.raises(ValueError, match="share memory"):
            lib.kv_read(*args, out=pair)
    assert not bool(both.any())
    got, want = lib.kv_read(*args, out=(both[20:], both[:20])), lib.kv_read(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
