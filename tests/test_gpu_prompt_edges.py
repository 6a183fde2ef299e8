"""attend_prompt where its inputs' strides, sizes and weights are at their ends."""
import pytest

from tests.prompt_ref import check, lens_to_cu, make, ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,strides", [
    ((1, 2, 64), (7, 64, 1)), ((40, 1, 64), (64, 5, 1)), ((1, 1, 128), (3, 5, 1)), ((1, 2, 64), (1 << 24, 64, 1)),
])
def test_any_stride_of_a_dimension_of_one(lib, shape, strides):
    """Tensors off 16 bytes are copied, whatever the strides are that their dimensions of size 1 carry."""
    import torch
    n, h, d = shape
    data = [x.cuda() for x in make(3, [n], [n], h, h, d, torch.bfloat16)]
    cu = lens_to_cu([n])
    want = ref(*[x.cpu() for x in data[:3]], cu, cu, d ** -0.5, 0, data[3].cpu())

    def lay(x):
        flat = torch.zeros(x.numel() + 8, device="cuda", dtype=x.dtype)
        return flat.as_strided(shape, strides, 1).copy_(x)
    leaves = [lay(x).detach().requires_grad_() for x in data[:3]]
    assert leaves[0].stride() == strides and leaves[0].data_ptr() % 16 != 0
    out = lib.attend_prompt(*leaves, cu.cuda())
    got = (out,) + torch.autograd.grad(out, leaves, lay(data[3]))
    for name, x in zip(("out", "dq", "dk", "dv"), got):
        check(name, x, want[name])


def test_a_head_dim_past_32_bits_is_refused(lib):
    import torch
    q = torch.empty(0, 1, (1 << 32) + 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="too large"):
        lib.attend_prompt(q, q, q, cu)
