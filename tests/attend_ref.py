"""Plain fp64 forms of the paged e4m3 cache's operators (CPU torch), their
inputs, and the tolerance of an attention output.

Tolerance of out = sum_s w_s v_s / sum_s w_s against fp64, with
A = sum_s w_s |v_s| / sum_s w_s and n visible keys:
  2^-8 |out|     the output's rounding to bf16 (half a step);
  2^-11 A        each weight's rounding to fp16;
  2 E A          the score's fp32 error E in the weight, in numerator and
                 divisor: D + 4 roundings of 2^-24 on sum_d |q_d k_d| scale,
                 8 of 2^-24 on the scores' and log2(v_scale)'s size, and
                 2^-22 for 2^x and 1 / v_scale;
  2 n 2^-24 A    n fp32 additions, in numerator and divisor;
  n 2^-25 448 vs weights below fp16's normal range (absolute 2^-25 of the
                 largest, which is at least 1; vs the largest value scale).
"""
from __future__ import annotations

import torch

E4M3_MAX = 448.0


def make_cache(gen, n_pages, Hkv, page, D, pow2=True, spread=1.0):
    """(k, v, k_scale, v_scale) on the CPU; every byte finite."""
    def one():
        x = torch.randn(n_pages, Hkv, page, D, generator=gen)
        amp = torch.exp2(spread * torch.randn(n_pages, Hkv, generator=gen))
        s = amp * x.abs().amax((2, 3)) / E4M3_MAX
        if pow2:
            s = torch.exp2(torch.ceil(torch.log2(s)))
        b = (x * (amp / s)[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return b, s
    k, ks = one()
    v, vs = one()
    return k, v, ks, vs


def make_batch(gen, rows, lens, page, spare=2, max_pages=None):
    """page_table, cu, kv_len (CPU int32) with every page id used at most once,
    and the number of pages; unused table entries hold -1."""
    B = len(rows)
    need = [max(0, -(-n // page)) for n in lens]
    mp = max_pages or max(1, max(need + [0]))
    ids = torch.randperm(sum(need) + spare, generator=gen)
    table = torch.full((B, mp), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = min(need[b], mp)
        table[b, :n] = ids[at:at + n].int()
        at += need[b]
    cu = torch.tensor([0] + rows).cumsum(0).int()
    return table, cu, torch.tensor(lens, dtype=torch.int32), sum(need) + spare


def poison(cache, table, lens, page, window_lo=None):
    """NaN bytes and scales wherever no token of a sequence lives."""
    k, v, ks, vs = cache
    used = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for p in range(-(-max(n, 0) // page)):
            if p < table.shape[1] and 0 <= int(table[b, p]) < k.shape[0]:
                used[int(table[b, p]), :min(page, n - p * page)] = True
    for x in (k, v):
        x.view(torch.uint8).permute(0, 2, 1, 3)[~used] = 0x7F
    for s in (ks, vs):
        s[~used.any(1)] = float("nan")


def dense_kv(cache, table_row, n, page):
    """k, v [Hkv, n, D] fp64 of a sequence's first n tokens and ok [n]: the token has a page."""
    k, v, ks, vs = cache
    s = torch.arange(n)
    pg = s // page
    ok = pg < table_row.shape[0]
    ids = table_row[pg.clamp(max=table_row.shape[0] - 1)].long()
    ok &= (ids >= 0) & (ids < k.shape[0])
    ids = torch.where(ok, ids, 0)
    get = lambda x, sc: x.view(torch.uint8)[ids, :, s % page].view(torch.float8_e4m3fn).double() * sc[ids].double()[..., None]
    kk, vv = get(k, ks), get(v, vs)
    zero = ~ok[:, None, None]
    return kk.masked_fill(zero, 0).transpose(0, 1), vv.masked_fill(zero, 0).transpose(0, 1), ok


def softmax_rows(q, k, v, see, scale, vs_max):
    """One row: q [Hq, D], k, v [Hkv, n, D] fp64, see [n].  (out, tol) [Hq, D]."""
    Hq, D = q.shape
    G = Hq // k.shape[0]
    n = int(see.sum())
    if n == 0:
        return torch.zeros(Hq, D, dtype=torch.float64), torch.zeros(Hq, D, dtype=torch.float64)
    k, v = k[:, see].repeat_interleave(G, 0), v[:, see].repeat_interleave(G, 0)
    qd = q.double()[:, None]
    x = (qd * k).sum(-1) * scale
    w = torch.softmax(x, -1)[..., None]
    out, A = (w * v).sum(1), (w * v.abs()).sum(1)
    size = ((qd * k).abs().sum(-1) * abs(scale)).amax(-1, keepdim=True)
    E = (D + 4) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * (size + 64) + 2.0 ** -22
    tol = 2.0 ** -8 * out.abs() + (2.0 ** -11 + 2 * E + n * 2.0 ** -23) * A + n * 2.0 ** -25 * E4M3_MAX * vs_max
    return out, tol


def ref_attend(q, cache, table, cu, kv_len, scale, window=0, n_sink=0, idx=None):
    """out, tol [T, Hq, D] fp64 and written [T]."""
    T, Hq, D = q.shape
    page = cache[0].shape[2]
    out, tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    written = torch.zeros(T, dtype=torch.bool)
    vs_max = float(torch.nan_to_num(cache[3], nan=0.0).max())
    for b in range(table.shape[0]):
        r0, r1 = int(cu[b]), int(cu[b + 1])
        n = int(kv_len[b])
        k, v, ok = dense_kv(cache, table[b], max(n, 0), page)
        key = torch.arange(max(n, 0))
        for r in range(r0, r1):
            pos = n - (r1 - r0) + (r - r0)
            see = ok & (key <= pos)
            if window > 0:
                see &= (key > pos - window) | (key < n_sink)
            kk, vv = k, v
            if idx is not None:
                e = idx[r].long()
                e = e[(e >= 0) & (e < n)]
                kk, vv, see = k[:, e], v[:, e], see[e]
            out[r], tol[r] = softmax_rows(q[r], kk, vv, see, scale, vs_max)
            written[r] = True
    return out, tol, written


def ref_packed(q, cache, table, kv_len, shared, masks, lens, group, scale):
    T = q.shape[0]
    n, page = int(kv_len[0]), cache[0].shape[2]
    k, v, ok = dense_kv(cache, table[0], max(n, 0), page)
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    vs_max = float(torch.nan_to_num(cache[3], nan=0.0).max())
    m = masks.view(torch.int32)
    for t in range(T):
        g, pos = t // group, n - T + t
        length = min(max(int(lens[g]), 0), shared.shape[1])
        e = shared[g, :length].long()
        e = e[((m[g, :length] >> (t % group)) & 1) != 0]
        e = e[(e >= 0) & (e <= pos) & (e < n)]
        out[t], tol[t] = softmax_rows(q[t], k[:, e], v[:, e], ok[e], scale, vs_max)
    return out, tol


def pow2_scale(amax):
    """Least power of two s with amax <= 448 s, in [2^-64, 2^64]."""
    m, e = torch.frexp(amax.double())
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 64)
    return torch.exp2(torch.where(amax > 0, e, -64).double()).float()


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, D] fp64 rotated by positions pos [T]."""
    half = inv_freq.shape[0]
    ang = pos.double()[:, None, None] * inv_freq
    i = torch.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = x.clone()
    y[..., lo] = x[..., lo] * torch.cos(ang) - x[..., hi] * torch.sin(ang)
    y[..., hi] = x[..., hi] * torch.cos(ang) + x[..., lo] * torch.sin(ang)
    return y


def ref_append(k, v, cache, table, cu, kv_len, inv_freq, interleaved):
    """The cache after the append (new tensors)."""
    page, n_pages = cache[0].shape[2], cache[0].shape[0]
    data = [cache[0].clone(), cache[1].clone()]
    scale = [cache[2].clone(), cache[3].clone()]
    for b in range(table.shape[0]):
        r0, r1, n = int(cu[b]), int(cu[b + 1]), max(int(kv_len[b]), 0)
        pos = torch.arange(n - (r1 - r0), n)
        kr = k[r0:r1].double()
        if inv_freq is not None:
            kr = rotate(kr, pos, inv_freq, interleaved)
        for d, sc, x in ((data[0], scale[0], kr.float()), (data[1], scale[1], v[r0:r1].float())):
            for p in sorted(set((pos[pos >= 0] // page).tolist())):
                if p >= table.shape[1] or not 0 <= int(table[b, p]) < n_pages:
                    continue
                pid = int(table[b, p])
                rows = (pos // page == p) & (pos >= 0)
                slot = int(pos[rows][0]) % page
                y = x[rows].transpose(0, 1)
                s = pow2_scale(y.abs().amax((1, 2)))
                if slot:
                    s = torch.maximum(s, sc[pid])
                    old = d[pid, :, :slot].float() * (sc[pid] / s)[:, None, None]
                    moved = old.to(torch.float8_e4m3fn).view(torch.uint8)
                    keep = (s == sc[pid])[:, None, None]
                    d.view(torch.uint8)[pid, :, :slot] = torch.where(keep, d.view(torch.uint8)[pid, :, :slot], moved)
                q = (y / s[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                d.view(torch.uint8)[pid, :, slot:slot + int(rows.sum())] = q.view(torch.uint8)
                sc[pid] = s
    return data[0], data[1], scale[0], scale[1]
