"""A run of the prompts' operators as they would be used: a prompt is attended
whole and stored, several answers share it, one of them is read back and
continued in 16 bits, with the gradient."""
import pytest

from tests.attend_ref import ref_append, ref_attend
from tests.prompt_ref import check, lens_to_cu, ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_answers_and_next_turn(lib, D):
    import torch
    n, B, steps, Hq, Hkv, page = 150, 5, 3, 8, 2, 32
    g = torch.Generator().manual_seed(D)
    r = lambda t, h: torch.randn(t, h, D, generator=g).bfloat16()
    scale = D ** -0.5
    per = -(-(n + steps + 40) // page)
    pool = B * per + 1
    cache = tuple(torch.zeros(pool, Hkv, page, D, dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)) + \
        tuple(torch.ones(pool, Hkv) for _ in range(2))
    c = [x.clone().cuda() for x in cache]
    ids = torch.randperm(pool, generator=g).int()
    table = torch.stack([ids[b * per:(b + 1) * per] for b in range(B)])

    # the prompt: attended in 16 bits, its keys and values stored
    q, k, v = r(n, Hq), r(n, Hkv), r(n, Hkv)
    cu = lens_to_cu([n])
    out, lse = lib.attend_prompt(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), return_lse=True)
    want = ref(q, k, v, cu, cu, scale)
    check("out", out, want["out"]), check("lse", lse, want["lse"])
    kv_len = torch.tensor([n], dtype=torch.int32)
    lib.kv_append(k.cuda(), v.cuda(), c, table[:1].cuda(), cu.cuda(), kv_len.cuda())
    cache = ref_append(k, v, cache, table[:1], cu, kv_len, None, False)
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c, cache))

    # the answers share the prompt's whole pages; the page that it ends in is copied
    whole = n // page
    table[:, :whole] = table[0, :whole]
    for b in range(1, B):
        for x in (cache, c):
            for t in x:
                t.view(torch.uint8)[int(table[b, whole])] = t.view(torch.uint8)[int(table[0, whole])]
    groups, shared = torch.tensor([0, B], dtype=torch.int32), torch.tensor([n], dtype=torch.int32)
    cu = lens_to_cu([1] * B)
    for s in range(steps):
        q, k, v = r(B, Hq), r(B, Hkv), r(B, Hkv)
        kv_len = torch.full((B,), n + s + 1, dtype=torch.int32)
        args = [x.cuda() for x in (table, cu, kv_len)]
        lib.kv_append(k.cuda(), v.cuda(), c, *args)
        cache = ref_append(k, v, cache, table, cu, kv_len, None, False)
        # (a page's scale that moves would move the shared keys' bytes in that sequence's copy: tokens
        # of a page that is no sequence's alone are shared up to the page)
        shared[0] = whole * page
        out = lib.attend_shared(q.cuda(), c, *args, groups.cuda(), shared.cuda())
        val, tol, _ = ref_attend(q, cache, table, cu, kv_len, scale)
        assert bool(((out.cpu().double() - val).abs() <= tol).all())

    # the third answer is read back and its next turn attended over it in 16 bits, with gradients
    turn, m = 33, n + steps
    one = [x.cuda() for x in (table[2:3], lens_to_cu([m]), torch.tensor([m], dtype=torch.int32))]
    kh, vh = lib.kv_read(c, *one, m)
    q, k, v, dout = r(turn, Hq), r(turn, Hkv), r(turn, Hkv), r(turn, Hq)
    keys, values = (torch.cat([a.cpu(), b]) for a, b in ((kh, k), (vh, v)))
    cu, ck = lens_to_cu([turn]), lens_to_cu([m + turn])
    leaves = [x.cuda().requires_grad_() for x in (q, keys, values)]
    out = lib.attend_prompt(*leaves, cu.cuda(), ck.cuda())
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(out, leaves, dout.cuda())), out=out)
    want = ref(q, keys, values, cu, ck, scale, 0, dout)
    for name, x in got.items():
        check(name, x, want[name])
