"""Appending to pages whose scale another writer chose: bytes rounded once to
e4m3, also where the scale is no power of two and the quotient lies within
2^-24 of a border between two bytes."""
import bisect
from fractions import Fraction

import pytest

from tests.gpu_util import say
from tests.test_gpu_attend import _dev, _gen

pytestmark = pytest.mark.gpu


def _table():
    """The finite e4m3 magnitudes in order (byte b is entry b)."""
    import torch
    return [Fraction(x) for x in torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double().tolist()]


def _nearest(x, vals):
    """Byte of the e4m3 value nearest to the fraction x, ties to the even byte, saturated."""
    m = abs(x)
    i = min(bisect.bisect_left(vals, m), len(vals) - 1)
    if i > 0 and (m - vals[i - 1] < vals[i] - m or (m - vals[i - 1] == vals[i] - m and (i - 1) % 2 == 0)):
        i -= 1
    return i | (0x80 if x < 0 else 0)


def _borders(vals):
    """Midpoints of neighbouring normal values, one of each 4-bit pattern."""
    return [(vals[b] + vals[b + 1]) / 2 for b in range(0x38, 0x38 + 16)]


def _near(x):
    """The fp32 numbers around the fraction x, as fractions."""
    import torch
    f = torch.tensor(float(x), dtype=torch.float64).float()
    return [Fraction(torch.nextafter(f, f.new_tensor(t)).item()) if t else Fraction(f.item()) for t in (0, float("inf"), 0.0)]


def _run(lib, olds, rows, held, D=64, page=16, slot=3):
    """One sequence a page whose first `slot` tokens hold the bytes `held` under the scales `olds`; appends `rows`
    [B, D] (bf16 values) to keys and values of the one head.  Returns keys' bytes and scales, values' the same."""
    import torch
    B = len(olds)
    kb = torch.zeros(B, 1, page, D, dtype=torch.uint8)
    kb[:, 0, :slot] = held[:, None]
    ks = torch.tensor([[float(o)] for o in olds], dtype=torch.float64).float()
    cache = _dev(kb.view(torch.float8_e4m3fn), kb.clone().view(torch.float8_e4m3fn), ks, ks.clone())
    x = rows.bfloat16()
    assert torch.equal(x.double(), rows)
    x = x[:, None].contiguous().cuda()
    lib.kv_append(x, x, cache, torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                  torch.arange(B + 1, dtype=torch.int32, device="cuda"), torch.full((B,), slot + 1, dtype=torch.int32, device="cuda"))
    return [t.cpu() for t in cache]


def test_rows_joining_a_page_of_another_scale(lib):
    """Values x = midpoint times scale, for scales next to x / midpoint on both sides: the quotient is off the border by
    less than 2^-23 of itself, and rounds to the side that it is on."""
    import torch
    vals, g = _table(), _gen(91)
    olds, xs = [], []
    for m in _borders(vals):
        for t in (129, 163, 201, 255):              # bf16 values of 8 bits
            for s in _near(Fraction(t, 64) / m):
                olds.append(s), xs.append(Fraction(t, 64))
    B = len(olds)
    rows = torch.randn(B, 64, generator=g).bfloat16().double()
    rows[:, 5] = torch.tensor([float(x) for x in xs], dtype=torch.float64)
    rows[:, 6] = -rows[:, 5]
    held = torch.randint(0, 0x7F, (B, 64), generator=g, dtype=torch.uint8)
    k, v, ks, vs = _run(lib, olds, rows, held)
    say("joining", B)
    assert [Fraction(x) for x in ks[:, 0].double().tolist()] == olds       # none grows: |x| <= 4 < 448 scale
    want = torch.tensor([[_nearest(Fraction(x) / o, vals) for x in r] for o, r in zip(olds, rows.tolist())], dtype=torch.uint8)
    for t in (k, v):
        got = t.view(torch.uint8)[:, 0]
        assert torch.equal(got[:, 0], held) and torch.equal(got[:, 2], held) and not got[:, 4:].any()
        # (a zero keeps its sign or not: the same value)
        d = (got[:, 3] != want) & ((got[:, 3] | want) != 0x80)
        assert not d.any(), f"{int(d.sum())} of {d.numel()} bytes differ"


def test_tokens_of_a_page_whose_other_scale_grows(lib):
    """Bytes times scale within 2^-23 of a border of the grown scale (a power of two)."""
    import torch
    vals, g = _table(), _gen(92)
    olds, bytes_ = [], []
    for m in _borders(vals):
        for b in (0x39, 0x3B, 0x3D, 0x3F):          # 9/8, 11/8, 13/8, 15/8
            for s in _near(m / vals[b]):
                olds.append(s), bytes_.append(b)
    B = len(olds)
    held = torch.randint(0, 0x7F, (B, 64), generator=g, dtype=torch.uint8)
    held[:, 5] = torch.tensor(bytes_, dtype=torch.uint8)
    held[:, 6] = held[:, 5] | 0x80
    rows = torch.zeros(B, 64, dtype=torch.float64)
    rows[:, 7] = 448.0 * 8                            # the scale becomes 8: products lie between 2^-3 and 1/2 of the border
    olds = [8 * o for o in olds]                      # .. and olds above 8 stay
    grown = [max(o, Fraction(8)) for o in olds]
    k, v, ks, vs = _run(lib, olds, rows, held)
    say("growing", B)
    assert [Fraction(x) for x in ks[:, 0].double().tolist()] == grown
    want = torch.tensor([[_nearest(vals[b & 0x7F] * (-1 if b & 0x80 else 1) * o / n, vals) for b in r] if n > o else r
                         for o, n, r in zip(olds, grown, held.tolist())], dtype=torch.uint8)
    assert sum(n > o for o, n in zip(olds, grown)) > 20
    for t in (k, v):
        got = t.view(torch.uint8)[:, 0]
        for slot in range(3):
            d = (got[:, slot] != want) & ((got[:, slot] | want) != 0x80)
            assert not d.any(), f"{int(d.sum())} of {d.numel()} bytes differ"


def _pi():
    """pi to 70 digits: 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inv(n, one):
        t = s = one // n
        k = 1
        while t:
            t //= n * n
            k += 2
            s += -t // k if k % 4 == 3 else t // k
        return s
    one = 10 ** 80
    return Fraction(16 * atan_inv(5, one) - 4 * atan_inv(239, one), one)


@pytest.mark.parametrize("pos,f", [(1048575, 3.0 ** 33), (2 ** 31 - 129, 3.0 ** 26), (777777, 2.0 ** 50 + 1), (999, 5.0 ** 22)])
def test_rotation_by_many_turns(lib, pos, f):
    """Angles of up to 2^72 radians: 1 / 2pi takes both words of its constant.  The reduced angle is off by the third
    word (2^-109 of the angle in turns) and the products' roundings (2^-35 turns): neither reaches a byte's border here
    nor a bf16's half step."""
    import math
    import torch
    g = _gen(93)
    pi, D, page = _pi(), 64, 16
    assert abs(float(pi) - math.pi) < 1e-15
    freq = torch.tensor([f / (i + 1) for i in range(32)], dtype=torch.float64)
    turns = [(pos * Fraction(x) / (2 * pi)) % 1 for x in freq.tolist()]
    ang = torch.tensor([float(2 * pi * t) for t in turns], dtype=torch.float64)
    x = torch.randn(1, 2, D, generator=g).bfloat16()
    lo, hi = x.double()[..., :32], x.double()[..., 32:]
    ref = torch.cat([lo * ang.cos() - hi * ang.sin(), hi * ang.cos() + lo * ang.sin()], -1)
    zero = torch.zeros(1, 2, page, D, dtype=torch.uint8)
    cache = _dev(zero.view(torch.float8_e4m3fn), zero.clone().view(torch.float8_e4m3fn), torch.ones(1, 2), torch.ones(1, 2))
    table = torch.zeros(1, pos // page + 1, dtype=torch.int32)
    say("turns", pos, f)
    q = lib.kv_append(*_dev(x, x), cache, *_dev(table, torch.tensor([0, 1]).int(), torch.tensor([pos + 1]).int(), freq, x))
    tol = 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -24 * 2 * x.double().abs().amax(-1, keepdim=True)
    assert ((q.cpu().double() - ref).abs() <= tol).all()
    s = cache[2].cpu().double()[0][:, None]
    want = (ref[0] / s).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(cache[0].cpu().view(torch.uint8)[0, :, pos % page], want)
