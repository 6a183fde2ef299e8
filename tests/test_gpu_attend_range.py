"""The paged e4m3 cache's attention at the ends of the value scales' range,
2^-64 and 2^64 in one sequence (a page of zeros is written with 2^-64), by every
kernel: few and many rows a key, lists, packed groups, whole and cut units."""
import math

import pytest

from tests.attend_ref import E4M3_MAX, make_batch
from tests.gpu_util import say
from tests.test_gpu_attend import _dev, _gen, _within
from tests.test_gpu_attend_edges import _widen

pytestmark = pytest.mark.gpu

# order of the pages of small scales among the others
ORDERS = {"first": lambda p, n: p < n // 2, "last": lambda p, n: p >= n // 2, "in turn": lambda p, n: p % 2 == 0,
          "one": lambda p, n: p == n // 3}


def _far_apart(T, L, Hkv, G, D, order, shift, zero, seed):
    """Pages with value scales 2^-64 and 2^64; scores of the small pages' keys are `shift` higher in base 2.  Value bytes
    are large and positive, or zero in the small pages."""
    import torch
    g = _gen(seed)
    page = 16
    table, cu, n, pages = make_batch(g, [T], [L], page)
    small = torch.zeros(pages, dtype=torch.bool)
    used = -(-L // page)
    for p in range(used):
        small[int(table[0, p])] = ORDERS[order](p, used)
    k = torch.zeros(pages, Hkv, page, D)
    k[..., 0] = 1.0
    v = 256.0 + 16 * torch.randint(0, 12, (pages, Hkv, page, D), generator=g)
    if zero:
        v[small] = 0.0
    ks = torch.where(small, float(abs(shift)), 1.0)[:, None].repeat(1, Hkv)
    k[small] *= math.copysign(1.0, shift) if shift else 0.0
    k[~small] = 0.0
    ks = ks.clamp(min=1.0)
    vs = torch.where(small, 2.0 ** -64, 2.0 ** 64)[:, None].repeat(1, Hkv)
    cache = (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), ks, vs)
    q = torch.zeros(T, Hkv * G, D)
    q[..., 0] = 1.0
    return cache, table, cu, n, q.bfloat16(), small[table[0].long()][torch.arange(L) // page]


def _sums(cache, table, small, T, L, G, lo, shift):
    """out and its tolerance [T, Hq, D] for rows that see the keys from lo to their own, in closed form: keys of small
    pages weigh 2^shift, the others 1.  The tolerance is attend_ref.py's, with two roundings of a weight to fp16 and
    weights below fp16's normal range off by 2^-25 of the row's largest weight times value scale."""
    import torch
    Hkv, page, D = cache[1].shape[1:]
    key = torch.arange(lo, L)
    byte = cache[1].view(torch.uint8)[table[0, key // page].long(), :, key % page].view(torch.float8_e4m3fn).double()
    sm = small[lo:].double()[:, None, None]
    rows = torch.arange(L - T - lo, L - lo)
    Ws, Wb = (sm.cumsum(0) * 2.0 ** shift)[rows], (1 - sm).cumsum(0)[rows]
    vs, vb = 2.0 ** (shift - 64), 2.0 ** 64
    out = ((byte * sm).cumsum(0)[rows] * vs + (byte * (1 - sm)).cumsum(0)[rows] * vb) / (Ws + Wb)
    top = torch.maximum((Ws > 0) * vs, (Wb > 0) * vb)
    size = abs(shift) * math.log(2.0)
    E = (D + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * (size + 64) + 2.0 ** -22
    n = len(key)
    tol = (2.0 ** -8 + 2.0 ** -10 + 2 * E + n * 2.0 ** -23) * out + n * 2.0 ** -25 * E4M3_MAX * top / (Ws + Wb)
    return out.repeat_interleave(G, 1), tol.repeat_interleave(G, 1)


SHIFTS = [0, 5, -7, 60, 127, 140]


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("T,L,G,D,log2_work", [
    (1, 64, 1, 64, 0), (1, 64, 2, 128, 0),              # one wave
    (1, 400, 4, 128, 0), (9, 700, 4, 64, 0),             # several waves; units of 32 rows
    (1, 9000, 4, 64, 0), (20, 9000, 8, 128, 0),          # cut units
    (80, 300, 4, 64, 24), (80, 300, 4, 128, 24),         # units of 128 rows
    (140, 2000, 4, 64, 25), (140, 2000, 4, 128, 25),     # units of 256 rows, cut
])
def test_value_scales_at_the_ends_of_their_range(lib, T, L, G, D, log2_work, order):
    for shift in SHIFTS:
        for zero in (False, True):
            say("range", T, L, G, D, order, shift, zero)
            cache, table, cu, n, q, small = _far_apart(T, L, 2, G, D, order, shift, zero, 81)
            if log2_work:
                table = _widen(table, 16, T, 2 * G, log2_work)
            out = lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n), scale=math.log(2.0))
            ref, tol = _sums(cache, table, small, T, L, G, 0, shift)
            _within(out, ref, tol, f"{order}, shift {shift}, zero {zero}")


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("T,L,G,D,topk", [(3, 64, 2, 64, 64), (2, 700, 17, 128, 500), (2, 6000, 4, 64, 5000)])
def test_value_scales_at_the_ends_of_their_range_selected(lib, T, L, G, D, topk, order):
    import torch
    for shift in SHIFTS:
        cache, table, cu, n, q, small = _far_apart(T, L, 2, G, D, order, shift, False, 82)
        idx = torch.arange(L - topk, L).repeat(T, 1).int()
        say("range, selected", T, L, G, D, order, shift)
        out = lib.attend_selected(q.cuda(), _dev(*cache), *_dev(table, cu, n, idx), scale=math.log(2.0))
        ref, tol = _sums(cache, table, small, T, L, G, L - topk, shift)
        _within(out, ref, tol, f"{order}, shift {shift}")


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("T,L,G,D,group", [(5, 300, 2, 64, 5), (16, 900, 4, 128, 8), (33, 700, 4, 64, 32),
                                           (32, 700, 8, 128, 16), (16, 4000, 8, 64, 16)])
def test_value_scales_at_the_ends_of_their_range_packed(lib, T, L, G, D, group, order):
    import torch
    for shift in SHIFTS:
        cache, table, cu, n, q, small = _far_apart(T, L, 2, G, D, order, shift, False, 83)
        ng = -(-T // group)
        shared = torch.arange(L).repeat(ng, 1).int()
        masks = torch.full((ng, L), -1, dtype=torch.int32).view(torch.uint32)
        lens = torch.full((ng,), L, dtype=torch.int32)
        say("range, packed", T, L, G, D, group, order, shift)
        out = lib.attend_packed(q.cuda(), _dev(*cache), *_dev(table, n, shared, masks, lens), group, scale=math.log(2.0))
        ref, tol = _sums(cache, table, small, T, L, G, 0, shift)
        _within(out, ref, tol, f"{order}, shift {shift}")


# ----------------------------------- a reference that moves in a step's second half

# A late key's score in base 2, as the two bytes (sixteenths) that make it.
LATE = [(224, 4), (256, 8), (288, 4), (320, 8), (352, 4)]


def _late_reference(T, Hkv, G, D, late, tail):
    """64 keys of score 0; then 64 of which 16 .. 31 score 7 to 7.9 and have large values, and one of the second half
    scores 14 to 22 and has the value 0; then `tail` keys of score 0 and value 0.  All scores in base 2."""
    import torch
    g = _gen(84)
    L = 128 + tail
    table, cu, n, pages = make_batch(g, [T], [L], 64, spare=0)
    k, v = torch.zeros(L, Hkv, D), torch.zeros(L, Hkv, D)
    k[80:96, :, 0] = 112.0
    k[80:96, :, 1] = torch.randint(0, 15, (16, Hkv), generator=g).float()
    k[104, :, 0], k[104, :, 1] = late
    v[80:96] = 256.0 + 16 * torch.randint(0, 12, (16, Hkv, D), generator=g)
    v = v.to(torch.float8_e4m3fn).float()      # the values that the bytes stand for
    score = (k[..., 0] + k[..., 1]).double() / 16
    cache = [torch.zeros(pages, Hkv, 64, D) for _ in range(2)]
    for dst, src in zip(cache, (k, v)):
        for p in range(-(-L // 64)):
            x = src[64 * p:64 * p + 64].transpose(0, 1)
            dst[int(table[0, p]), :, :x.shape[1]] = x
    cache = [x.to(torch.float8_e4m3fn) for x in cache] + [torch.full((pages, Hkv), 1.0 / 16), torch.ones(pages, Hkv)]
    q = torch.zeros(T, Hkv * G, D)
    q[..., :2] = 1.0
    w = torch.exp2(score)

    def ref(see):
        """Rows that see the keys below see [T].  Off by half a step of bf16, two roundings of a weight to fp16, the
        scores' error E, n additions, and twice 2^-25 of the largest weight for each of the 16 values."""
        W = w.cumsum(0)[see - 1]
        out = ((w[..., None] * v.double()).cumsum(0)[see - 1] / W[..., None])
        size = float(score.max()) * math.log(2.0)
        E = (D + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * (size + 64) + 2.0 ** -22
        tol = (2.0 ** -8 + 2.0 ** -10 + 2 * E + L * 2.0 ** -23) * out
        tol = tol + 16 * 2.0 ** -24 * E4M3_MAX * (w.max() / W)[..., None]
        return out.repeat_interleave(G, 1), tol.repeat_interleave(G, 1)
    return tuple(cache), table, cu, n, q.bfloat16(), ref


@pytest.mark.parametrize("late", LATE, ids=lambda x: str(sum(x) / 16))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("log2_work", [24, 25])
def test_weights_before_a_late_reference(lib, D, late, log2_work):
    import torch
    T, G = 80, 4
    cache, table, cu, n, q, ref = _late_reference(T, 2, G, D, late, T)
    say("late reference", D, late, log2_work)
    out = lib.attend(q.cuda(), _dev(*cache), *_dev(_widen(table, 64, T, 2 * G, log2_work), cu, n), scale=math.log(2.0))
    _within(out, *ref(torch.arange(128, 128 + T) + 1), f"late reference, {sum(late) / 16}")


@pytest.mark.parametrize("late", LATE, ids=lambda x: str(sum(x) / 16))
@pytest.mark.parametrize("D", [64, 128])
def test_weights_before_a_late_reference_packed(lib, D, late):
    """Enough groups that their lists are not cut."""
    import torch
    T, G, group = 1024, 8, 16
    cache, table, cu, n, q, ref = _late_reference(T, 8, G, D, late, T)
    shared = torch.arange(128).repeat(T // group, 1).int()
    masks = torch.full(shared.shape, -1, dtype=torch.int32).view(torch.uint32)
    lens = torch.full((T // group,), 128, dtype=torch.int32)
    say("late reference, packed", D, late)
    out = lib.attend_packed(q.cuda(), _dev(*cache), *_dev(table, n, shared, masks, lens), group, scale=math.log(2.0))
    _within(out, *ref(torch.full((T,), 128)), f"late reference, packed, {sum(late) / 16}")
