"""attend_shared's errors."""
import pytest

from tests.test_gpu_shared import shared_case

pytestmark = pytest.mark.gpu


def test_a_small_workspace_names_the_size_function_of_the_call(lib):
    import torch
    q, cache, table, cu, kv_len, bounds, lens = shared_case(14, [(64, [(1, 100), (2, 120)])], 2, 4, 16, 64)
    d, args = [x.cuda() for x in cache], [x.cuda() for x in (table, cu, kv_len)]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match=r"workspace too small.*attend_shared_workspace_bytes"):
        lib.attend_shared(q.cuda(), d, *args, bounds.cuda(), lens.cuda(), workspace=ws)
    with pytest.raises(ValueError, match=r"workspace too small.*\battend_workspace_bytes"):
        lib.attend(q.cuda(), d, *args, workspace=ws[:16])
