"""Plain fp64 forms of attention over 16-bit prompts and of its gradient, their
inputs, and tolerances.

u is half a step of the type (bf16 2^-8, fp16 2^-11) relative to a value; in
fp16 a weight or score gradient below the normal range is off by up to 2^-25
(of the reference 1 that the largest weight reaches).  Per row, with its scores
x_s, weights P_s, n keys, and E the error of a score in fp32,
  E = (D + 8) 2^-24 (sum_d |q_d k_d| scale + |x| + |lse|) + 2^-22
(D products and sums, the factor scale log2(e), the subtraction, 2^x):
  out   u |out| + (u + 2 E + n 2^-23) sum_s P_s |v_s| [+ 2^-25 n max|v|]
  lse   E + n 2^-24 + 2^-22 |lse|
The backward pass forms P again (error 2 E relative), and from what the forward
pass returned delta = dout . (out + rest), where rest holds what rounding left
out of out, to u of itself, off by
  d = sum_d |dout_d| (tol(out)_d - (u - u^2) |out_d| + D 2^-24 |out_d|),
and dP = dout . v, off by D 2^-24 sum_d |dout_d v_d| =: p:
  dS    e_s = |dS_s| (u + 2 E + 2^-22) + P_s (d + p) [+ 2^-25]
  dq    u |dq| + scale sum_s (e_s + n 2^-23 |dS_s|) |k_s|
  dk    u |dk| + scale sum_i (e_s + N 2^-23 |dS_s|) |q_i|       over the N rows and heads
  dv    u |dv| + sum_i (P (u + 2 E + N 2^-23) [+ 2^-25]) |dout_i|
Everything + 2^-100: a weight below fp32's normal range, 2^-126, is 0 (scores 88
apart), which leaves out at most 2^16 products of it with values up to 2^10.
"""
from __future__ import annotations

import math

import torch


def lens_to_cu(lens, first=0):
    return (torch.tensor([0] + list(lens)).cumsum(0) + first).int()


def visible(n, m, window):
    """[n, m]: row i, at position m - n + i, sees key s."""
    p = m - n + torch.arange(n)[:, None]
    s = torch.arange(m)
    see = s <= p
    if window > 0:
        see &= s > p - window
    return see


def make(seed, rows, keys, Hq, Hkv, D, dtype, spread=1.0, before=0, behind=0):
    """Packed q, k, v, dout (CPU), with `before` and `behind` rows and keys outside every sequence."""
    g = torch.Generator().manual_seed(seed)
    T, S = before + sum(rows) + behind, before + sum(keys) + behind
    r = lambda n, h: (spread * torch.randn(n, h, D, generator=g)).to(dtype)
    return r(T, Hq), r(S, Hkv), r(S, Hkv), torch.randn(T, Hq, D, generator=g).to(dtype)


def ref(q, k, v, cu, cu_k, scale, window=0, dout=None):
    """Values and tolerances: dict of (value, tolerance), fp64, of out, lse and, with dout, dq, dk, dv."""
    dtype, D = q.dtype, q.shape[2]
    u = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    G = q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, out_t = torch.zeros_like(q), torch.zeros_like(q)
    lse, lse_t = torch.full(q.shape[:2], -math.inf, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    grads = {x: (torch.zeros_like(y), torch.zeros_like(y)) for x, y in (("dq", q), ("dk", k), ("dv", v))}
    for b in range(len(cu) - 1):
        r0, r1, k0, k1 = int(cu[b]), int(cu[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        see = visible(r1 - r0, k1 - k0, window)
        some = see.any(1)
        n = see.sum(1, keepdim=True).double()
        for h in range(q.shape[1]):
            qh, kh, vh = q[r0:r1, h], k[k0:k1, h // G], v[k0:k1, h // G]
            if qh.shape[0] == 0 or kh.shape[0] == 0:
                continue
            x = (qh @ kh.T * scale).masked_fill(~see, -math.inf)
            ls = torch.logsumexp(x, -1, keepdim=True)
            P = torch.where(see, torch.exp(x - torch.where(some[:, None], ls, 0.0)), 0.0)
            size = (qh.abs() @ kh.abs().T * abs(scale)).masked_fill(~see, 0).amax(-1, keepdim=True)
            E = (D + 8) * 2.0 ** -24 * (2 * size + torch.where(some[:, None], ls.abs(), 0.0)) + 2.0 ** -22
            o, A = P @ vh, P @ vh.abs()
            vmax = vh.abs().amax(0, keepdim=True)
            ot = u * o.abs() + (u + 2 * E + n * 2.0 ** -23) * A + tiny * n * vmax + tiny
            out[r0:r1, h], out_t[r0:r1, h] = o, ot
            lse[r0:r1, h] = ls[:, 0]
            lse_t[r0:r1, h] = torch.where(some, (E + n * 2.0 ** -24 + 2.0 ** -22 * ls.abs())[:, 0], 0.0)
            if dout is None:
                continue
            do = dout[r0:r1, h].double()
            dP = do @ vh.T
            dS = P * (dP - (do * o).sum(-1, keepdim=True))
            d = (do.abs() * (ot + (u * u - u + D * 2.0 ** -24) * o.abs())).sum(-1, keepdim=True)
            p = D * 2.0 ** -24 * (do.abs() @ vh.abs().T)
            e = dS.abs() * (u + 2 * E + 2.0 ** -22) + P * (d + p) + tiny * see
            N = G * max(1, r1 - r0)
            val, tol = grads["dq"]
            val[r0:r1, h] = dS @ kh * scale
            tol[r0:r1, h] = u * val[r0:r1, h].abs() + abs(scale) * (e + n * 2.0 ** -23 * dS.abs()) @ kh.abs() + tiny
            val, tol = grads["dk"]
            val[k0:k1, h // G] += dS.T @ qh * scale
            tol[k0:k1, h // G] += abs(scale) * (e + N * 2.0 ** -23 * dS.abs()).T @ qh.abs() + tiny
            val, tol = grads["dv"]
            val[k0:k1, h // G] += P.T @ do
            tol[k0:k1, h // G] += (P * (u + 2 * E + N * 2.0 ** -23) + tiny * see).T @ do.abs() + tiny
    for name in ("dk", "dv"):
        val, tol = grads[name]
        tol += u * val.abs()
    res = {"out": (out, out_t), "lse": (lse, lse_t)}
    if dout is not None:
        res.update(grads)
    return res


def check(name, got, want):
    """got within the tolerance of want = (value, tolerance), infinities equal."""
    val, tol = want
    got = got.detach().cpu().double()
    assert got.shape == val.shape, (name, got.shape, val.shape)
    same = (got == val) | ((got - val).abs() <= tol + 2.0 ** -100)
    if not bool(same.all()):
        bad = (~same).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{name}: {len(bad)} of {same.numel()} off; at {i} got {got[i]}, want {val[i]} +- {tol[i]}")
