"""The sparse step's plumbing without a GPU."""
import contextlib

import pytest


@pytest.mark.parametrize("Hkv,T", [(2, 3), (8, 256)])
def test_every_part_runs_on_the_tensors_device(monkeypatch, Hkv, T):
    """The selection takes the current device's stream: the step makes the device of its tensors current for all parts,
    and leaves the caller's afterwards."""
    import torch
    from indexer_topk_long_amd import sparse
    current, calls = [], []

    @contextlib.contextmanager
    def device_of(t):
        current.append(t)
        yield
        current.pop()

    def part(name, result):
        def run(*a, **k):
            calls.append((name, list(current)))
            return result
        return run

    q = torch.zeros(T, 2 * Hkv, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(torch.cuda, "device_of", device_of)
    monkeypatch.setattr(sparse, "score_select", part("select", "idx"))
    monkeypatch.setattr(sparse, "dsa_pack", part("pack", ("shared", "masks", "lens")))
    monkeypatch.setattr(sparse, "kv_append", part("append", "rotated"))
    monkeypatch.setattr(sparse, "attend_packed", part("attend", "out"))
    monkeypatch.setattr(sparse, "attend_selected", part("attend", "out"))
    got = sparse.sparse_step(q, q[:, :Hkv], q[:, :Hkv], (), torch.zeros(1, 4), torch.tensor([T], dtype=torch.int32), None,
                             torch.zeros(T, 64), None, 16)
    assert got == ("out", "idx") and not current
    assert [n for n, _ in calls] == (["select", "pack", "append", "attend"] if Hkv == 8 else ["select", "append", "attend"])
    assert all(len(c) == 1 and c[0] is q for _, c in calls)
