"""Sizes and places that the operators of the cache and of prompts refuse before any device call."""
import pytest

from tests.test_attend_abi import EINVAL, OK, P, _append, _attend
from tests.test_prompt_abi import _read, _shared, lib  # noqa: F401


@pytest.mark.parametrize("D,most", [(128, (1 << 28) - 16), (64, (1 << 29) - 32)])
def test_reads_of_2_to_the_32_threads(D, most):
    kw = dict(n_kv_heads=1, head_dim=D, n_seq=0)              # (no sequence: no launch)
    assert _read(T=most, **kw) == OK
    for T in (most + 1, 1 << 30, (1 << 31) - 256):
        assert _read(T=T, **kw) == EINVAL


@pytest.mark.parametrize("at", [0, 16, -16, 2 * 4 * 2 * 128 - 16, 16 - 2 * 4 * 2 * 128])
def test_reads_into_one_place_twice(at):
    """T 4, two heads, D 128: 2,048 bytes each in 16 bits, 4,096 in 32."""
    for type_ in (0, 1, 2):
        assert _read(ko=P, vo=P + at, type=type_, n_kv_heads=2) == EINVAL
    assert _read(ko=P, vo=P + 2048 + at % 2048, type=2, n_kv_heads=2) == EINVAL
    assert _read(ko=P, vo=P + at, T=0) == OK


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 200, (1 << 31) - 1])
def test_more_sequences_or_groups_than_can_be_numbered(n):
    """Their numbers are halved by sums of two and stepped through by 256 or 512, in 32 bits."""
    for call in (_append, _shared, _read, lambda **kw: _attend("attend", **kw), lambda **kw: _attend("selected", **kw)):
        assert call(n_seq=n, T=0) == EINVAL
    assert _shared(n_group=n, T=0) == EINVAL
    assert _shared(n_group=1 << 30, n_seq=1 << 30, T=0, wsb=1 << 40) == OK
