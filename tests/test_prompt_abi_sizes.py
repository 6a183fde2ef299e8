"""Sizes and places that the prompts' operators refuse before any device call."""
import pytest

from tests.test_attend_abi import EINVAL, OK
from tests.test_prompt_abi import _read, lib  # noqa: F401


@pytest.mark.parametrize("D,most", [(128, (1 << 28) - 16), (64, (1 << 29) - 32)])
def test_reads_of_2_to_the_32_threads(D, most):
    kw = dict(n_kv_heads=1, head_dim=D, n_seq=0)              # (no sequence: no launch)
    assert _read(T=most, **kw) == OK
    for T in (most + 1, 1 << 30, (1 << 31) - 256):
        assert _read(T=T, **kw) == EINVAL
