"""The operators of prompts beside the 8-bit key/value cache: real cases, their
plain forms and exact values.

A batch of prompts is q [T, Hq, D], k and v [S, Hkv, D] in 16 bits with cu
[B + 1] (rows) and cu_k [B + 1] (keys): sequence b owns the rows cu[b] ..
cu[b+1]-1, at the last positions of its keys cu_k[b] .. cu_k[b+1]-1.  The
cache and its batches are those of kv_append and attend: pages k and v
[n_pages, Hkv, page, D] in e4m3 with one fp32 scale per page and head,
(page_table [B, max_pages], cu [B + 1], kv_len [B]).

  attend_prompt    causal attention over whole prompts, packed, with a sliding
                   window where asked; and its gradient
  attend_shared    rows of many sequences that share their first tokens:
                   those are read once for all
  kv_read          the rows of the cache back in 16 or 32 bits
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ----------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt, odd sizes, seven heads per key/value head: launch latency
        dict(name="prompt-short", op="prompt", B=1, new=37, hist=0, ragged=False, Hq=14, Hkv=2, D=64, dtype="bf16",
             window=0, fused=False, lse=False),
        # a serving batch's prompts, ragged, as slices of one projection's output
        dict(name="prompt-packed", op="prompt", B=16, new=2039, hist=0, ragged=True, Hq=32, Hkv=8, D=128,
             dtype="bf16", window=0, fused=True, lse=False),
        # one long prompt
        dict(name="prompt-16k", op="prompt", B=1, new=16384, hist=0, ragged=False, Hq=64, Hkv=8, D=128, dtype="bf16",
             window=0, fused=True, lse=False),
        # a window layer over two prompts, fp16, with the log-sums
        dict(name="prompt-window", op="prompt", B=2, new=8111, hist=0, ragged=True, Hq=32, Hkv=4, D=64, dtype="fp16",
             window=1024, fused=False, lse=True),
        # short new turns of four conversations after histories of up to 8,000 tokens
        dict(name="prompt-continued", op="prompt", B=4, new=129, hist=8000, ragged=True, Hq=32, Hkv=8, D=128,
             dtype="bf16", window=0, fused=False, lse=False),
        # a training step over short packed sequences, one key/value head a query head
        dict(name="train-short", op="train", B=8, new=301, hist=0, ragged=True, Hq=8, Hkv=8, D=64, dtype="fp16",
             window=0, fused=True),
        # a training step over packed sequences
        dict(name="train-packed", op="train", B=8, new=2048, hist=0, ragged=True, Hq=32, Hkv=8, D=128, dtype="bf16",
             window=0, fused=True),
        # a training step over one long sequence
        dict(name="train-8k", op="train", B=1, new=8192, hist=0, ragged=False, Hq=32, Hkv=8, D=128, dtype="bf16",
             window=0, fused=False),
        # four answers to a short prompt: launch latency
        dict(name="shared-short", op="shared", groups=1, per=4, new=1, prefix=1000, own=90, ragged=True, Hq=16, Hkv=4,
             D=64, page=32),
        # 64 answers to one long prompt
        dict(name="shared-64", op="shared", groups=1, per=64, new=1, prefix=32768, own=1000, ragged=True, Hq=64,
             Hkv=8, D=128, page=64),
        # a conversation's last tokens read back: launch latency
        dict(name="read-tail", op="read", B=1, new=100, L=4133, ragged=False, Hkv=4, D=64, page=16, dtype="bf16"),
        # four long prompts read back
        dict(name="read-prompts", op="read", B=4, new=32768, L=32768, ragged=True, Hkv=8, D=128, page=64,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "shared", "shared", "read"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, Hkv=Hkv, D=D)
    if op in ("prompt", "train"):
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _log_int(rng, 1, 32)
        pairs = 10 ** 8 if op == "train" else 2 * 10 ** 8
        new = _log_int(rng, 1, max(2, min(8192 if op == "train" else 16384, int(math.sqrt(pairs / B)))))
        hist = rng.choice([0, 0, _log_int(rng, 1, 4000)])
        c.update(B=B, new=new, hist=min(hist, max(0, pairs // (B * new) - new)), ragged=B > 1,
                 dtype=rng.choice(["bf16", "bf16", "fp16"]), window=rng.choice([0, 0, _log_int(rng, 16, 4096)]),
                 fused=False)
        c["fused"] = c["hist"] == 0 and rng.random() < 0.5
        if op == "prompt":
            c["lse"] = rng.random() < 0.3
    elif op == "shared":
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        groups, per = rng.choice([1, 1, 2, 5, 8]), _log_int(rng, 2, 64)
        c.update(groups=groups, per=per, new=rng.choice([1, 1, 1, rng.randint(2, 8)]),
                 prefix=_log_int(rng, 16, (1 << 15) // groups), own=_log_int(rng, 8, 1000), ragged=True,
                 page=rng.choice([16, 32, 64, 128]))
    else:
        B = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, (1 << 17) // B)
        c.update(B=B, new=new, L=new + rng.choice([0, _log_int(rng, 1, 4000)]), ragged=B > 1,
                 page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    return c


def _dtype(case):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]


def _spread(n, most, ragged, step):
    """n lengths of up to `most`, fixed by the case; the first is the longest."""
    return [1 + int((most - 1) * ((b * step) % 1.0)) if b and ragged else most for b in range(n)]


def _prompt_lens(case):
    """(rows, keys) of every sequence."""
    rows = _spread(case["B"], case["new"], case["ragged"], 0.7548776662)
    hist = _spread(case["B"], case["hist"], case["ragged"], 0.6180339887) if case["hist"] else [0] * case["B"]
    return rows, [n + h for n, h in zip(rows, hist)]


def _shared_lens(case):
    """Prefix of every group; rows and tokens of every sequence."""
    g, B = case["groups"], case["groups"] * case["per"]
    prefix = _spread(g, case["prefix"], case["ragged"], 0.7548776662)
    rows = _spread(B, case["new"], case["ragged"], 0.3247179572)
    own_len = _spread(B, case["own"], case["ragged"], 0.6180339887)
    return prefix, rows, [prefix[b // case["per"]] + max(n, o) for b, n, o in zip(range(B), rows, own_len)]


def _read_lens(case):
    rows = _spread(case["B"], case["new"], case["ragged"], 0.7548776662)
    return rows, [n + case["L"] - case["new"] for n in rows]


def _pairs(case, n, m):
    """(row, key) pairs of n rows at the last of m positions."""
    first = m - n + 1   # keys of the first row
    w = case["window"]
    if w <= 0 or w >= m:
        return n * first + n * (n - 1) // 2
    short = max(0, min(n, w - first))   # rows that see fewer keys than the window
    return short * first + short * (short - 1) // 2 + (n - short) * w


def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "read":
        T = sum(_read_lens(case)[0])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * Hkv * D * 2 * (1 + size) + -(-T // case["page"]) * Hkv * 8, "flops": T * Hkv * D * 2}
    Hq = case["Hq"]
    if case["op"] == "shared":
        prefix, rows, toks = _shared_lens(case)
        T, per = sum(rows), case["per"]
        own_keys = [t - prefix[b // per] for b, t in enumerate(toks)]
        keys = sum(prefix) + sum(own_keys)
        pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(rows, toks))
        return {"bytes": T * Hq * D * 4 + keys * Hkv * D * 2 + -(-keys // case["page"]) * Hkv * 8,
                "flops": 4 * D * Hq * pairs}
    rows, keys = _prompt_lens(case)
    T, S = sum(rows), sum(keys)
    pairs = sum(_pairs(case, n, m) for n, m in zip(rows, keys))
    if case["op"] == "prompt":
        return {"bytes": T * Hq * D * 4 + S * Hkv * D * 4 + (T * Hq * 4 if case["lse"] else 0),
                "flops": 4 * D * Hq * pairs}
    # forward: q, k, v, out; backward: those and dout read, dq, dk, dv written
    return {"bytes": T * Hq * D * 12 + S * Hkv * D * 12 + 2 * T * Hq * 4, "flops": 14 * D * Hq * pairs}


# ---------------------------------------------------------------- inputs

def _pool(g, n, Hkv, page, D):
    """A pool's bytes and scales: normal values whose size varies by page and head."""
    x = torch.randn(n, Hkv, page, D, device="cuda", generator=g)
    x *= torch.exp2(0.5 * torch.randn(n, Hkv, 1, 1, device="cuda", generator=g))
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def _cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Hkv, D = case["Hkv"], case["D"]
    s = dict(case=case)
    if case["op"] in ("prompt", "train"):
        Hq, dt = case["Hq"], _dtype(case)
        rows, keys = _prompt_lens(case)
        T, S = sum(rows), sum(keys)
        if case["fused"]:   # one projection's output holds q, k and v
            x = torch.randn(T, Hq + 2 * Hkv, D, device="cuda", generator=g)
            x[:, :Hq] *= 1.5
            x = x.to(dt)
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            q = (1.5 * torch.randn(T, Hq, D, device="cuda", generator=g)).to(dt)
            k = torch.randn(S, Hkv, D, device="cuda", generator=g).to(dt)
            v = torch.randn(S, Hkv, D, device="cuda", generator=g).to(dt)
        s.update(q=q, k=k, v=v, rows=rows, keys=keys, cu=_cu(rows), cu_k=_cu(keys) if case["hist"] else None)
        if case["op"] == "train":
            s["dout"] = torch.randn(T, Hq, D, device="cuda", generator=g).to(dt)
            for name in ("q", "k", "v"):
                s[name].requires_grad_(True)
        return s
    page = case["page"]
    if case["op"] == "shared":
        prefix, rows, toks = _shared_lens(case)
        per, B = case["per"], len(rows)
        # a sequence's table begins with its group's pages; where the prefix ends inside a page, that page is
        # every sequence's own copy
        whole = [p // page for p in prefix]
        need = [-(-t // page) for t in toks]
        total, most = sum(whole) + sum(n - whole[b // per] for b, n in enumerate(need)), max(need)
        s["k"], s["k_scale"] = _pool(g, total + 3, Hkv, page, D)
        s["v"], s["v_scale"] = _pool(g, total + 3, Hkv, page, D)
        ids = torch.randperm(total + 3, device="cuda", generator=g)
        table = torch.zeros(B, most, device="cuda", dtype=torch.int64)
        at = 0
        for j in range(case["groups"]):
            seqs = range(j * per, (j + 1) * per)
            table[seqs[0]:seqs[-1] + 1, :whole[j]] = ids[at:at + whole[j]]
            at += whole[j]
            for b in seqs:
                table[b, whole[j]:need[b]] = ids[at:at + need[b] - whole[j]]
                at += need[b] - whole[j]
            first, off = int(table[seqs[0], whole[j]]), prefix[j] % page
            if off:
                rest = table[seqs[0] + 1:seqs[-1] + 1, whole[j]]
                for data, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
                    byte = data.view(torch.uint8)
                    scale[rest] = scale[first].clone()
                    byte[rest, :, :off] = byte[first, :, :off].clone()
        s.update(table=table.int(), cu=_cu(rows), kv_len=torch.tensor(toks, device="cuda").int(),
                 groups=(per * torch.arange(case["groups"] + 1, device="cuda")).int(),
                 shared_len=torch.tensor(prefix, device="cuda").int(), prefix=prefix, rows=rows, toks=toks)
        s["q"] = (1.5 * torch.randn(sum(rows), case["Hq"], D, device="cuda", generator=g)).bfloat16()
        return s
    rows, toks = _read_lens(case)
    need = [-(-t // page) for t in toks]
    total = sum(need)
    s["k"], s["k_scale"] = _pool(g, total + 3, Hkv, page, D)
    s["v"], s["v_scale"] = _pool(g, total + 3, Hkv, page, D)
    ids = torch.randperm(total + 3, device="cuda", generator=g)
    table = torch.zeros(case["B"], max(need), device="cuda", dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    s.update(table=table.int(), cu=_cu(rows), kv_len=torch.tensor(toks, device="cuda").int(), rows=rows, T=sum(rows))
    return s


# ----------------------------------------------------------- plain forms

def _pad(x, lens, n):
    """[sum(lens), H, D] packed -> fp32 [H, B, n, D] padded with zeros."""
    if len(lens) == 1:
        return x.float()[None].permute(2, 0, 1, 3)
    out = torch.zeros(len(lens), n, *x.shape[1:], device="cuda")
    at = torch.tensor(lens, device="cuda")
    out[torch.arange(n, device="cuda")[None] < at[:, None]] = x.float()
    return out.permute(2, 0, 1, 3)


def _packed(x, lens):
    """[H, B, n, D] -> [sum(lens), H, D], the inverse of _pad."""
    x = x.permute(1, 2, 0, 3)
    if len(lens) == 1:
        return x[0]
    at = torch.tensor(lens, device="cuda")
    return x[torch.arange(x.shape[1], device="cuda")[None] < at[:, None]]


def _hidden(case, rows, keys):
    """[B, n, m]: the row does not see the key."""
    n, m = max(rows), max(keys)
    first = torch.tensor([b - a for a, b in zip(rows, keys)], device="cuda")[:, None, None]
    p = first + torch.arange(n, device="cuda")[None, :, None]
    s = torch.arange(m, device="cuda")
    hide = s > p
    if case["window"] > 0:
        hide |= s <= p - case["window"]
    return hide


def _prompt(s):
    c = s["case"]
    rows, keys, D, dt = s["rows"], s["keys"], c["D"], _dtype(c)
    B, G, n, scale = c["B"], c["Hq"] // c["Hkv"], max(s["rows"]), c["D"] ** -0.5
    q, k, v = _pad(s["q"].detach(), rows, n), _pad(s["k"].detach(), keys, max(keys)), _pad(s["v"].detach(), keys, max(keys))
    hide = _hidden(c, rows, keys)
    train = c["op"] == "train"
    if train:
        do = _pad(s["dout"], rows, n)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3] + (1,), device="cuda")
    for h in range(c["Hkv"]):
        kt = k[h].transpose(1, 2).contiguous()
        if train:
            dkh, dvh = torch.zeros_like(k[h]), torch.zeros_like(v[h])
        for x in range(h * G, (h + 1) * G):
            p = torch.bmm(q[x], kt).mul_(scale).masked_fill_(hide, float("-inf"))
            top = p.amax(-1, keepdim=True)
            p = p.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            out[x] = torch.bmm(p, v[h].contiguous()) / total
            lse[x] = top + torch.log(total)
            if train:
                p /= total
                dvh += torch.bmm(p.transpose(1, 2).contiguous(), do[x].contiguous())
                dp = torch.bmm(do[x].contiguous(), v[h].transpose(1, 2).contiguous())
                dp = dp.sub_((do[x] * out[x]).sum(-1, keepdim=True)).mul_(p).mul_(scale)
                dq[x] = torch.bmm(dp, k[h].contiguous())
                dkh += torch.bmm(dp.transpose(1, 2).contiguous(), q[x].contiguous())
        if train:
            dk[h], dv[h] = dkh, dvh
    res = {"out": _packed(out, rows).to(dt)}
    if train:
        res.update(dq=_packed(dq, rows).to(dt), dk=_packed(dk, keys).to(dt), dv=_packed(dv, keys).to(dt))
    elif c["lse"]:
        res["lse"] = _packed(lse, rows)[..., 0]
    return res


def _dequantised(s, data, scale, table):
    """[B, Hkv, max_pages * page, D] fp32 of the pages of a table."""
    x = data[table].float() * scale[table][..., None, None]
    return x.transpose(1, 2).reshape(table.shape[0], data.shape[1], -1, data.shape[3])


def _shared(s):
    """The prefix's keys met once by all rows of its group, then every sequence's own keys."""
    c = s["case"]
    D, Hkv, page, per, n = c["D"], c["Hkv"], c["page"], c["per"], max(s["rows"])
    G, B = c["Hq"] // Hkv, len(s["rows"])
    q = _pad(s["q"], s["rows"], n).view(Hkv, G, B, n, D)
    table = s["table"].long()
    out = torch.empty(Hkv, G, B, n, D, device="cuda")
    for j, S in enumerate(s["prefix"]):
        b0, b1 = j * per, (j + 1) * per
        w = S // page   # the pages from here on are the sequences' own
        rows, toks = s["rows"][b0:b1], s["toks"][b0:b1]
        kp = _dequantised(s, s["k"], s["k_scale"], table[b0:b0 + 1, :-(-S // page)])[0, :, :S]
        vp = _dequantised(s, s["v"], s["v_scale"], table[b0:b0 + 1, :-(-S // page)])[0, :, :S]
        ko, vo = (_dequantised(s, a, b, table[b0:b1, w:]) for a, b in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
        pos = torch.tensor(toks, device="cuda")[:, None] - torch.tensor(rows, device="cuda")[:, None] + \
            torch.arange(n, device="cuda")
        key = w * page + torch.arange(ko.shape[2], device="cuda")
        hide = (key > pos[..., None]) | (key < S)                      # [per, n, own keys]
        qg = q[:, :, b0:b1]                                            # [Hkv, G, per, n, D]
        x = torch.bmm(qg.reshape(Hkv, -1, D), kp.transpose(1, 2).contiguous()).mul_(D ** -0.5).view(Hkv, G, per, n, S)
        qo = qg.permute(2, 0, 1, 3, 4).reshape(per * Hkv, G * n, D)
        y = torch.bmm(qo, ko.reshape(per * Hkv, -1, D).transpose(1, 2).contiguous()).mul_(D ** -0.5)
        y = y.view(per, Hkv, G, n, -1).masked_fill_(hide[:, None, None], float("-inf"))
        top = torch.maximum(x.amax(-1), y.amax(-1).permute(1, 2, 0, 3))     # [Hkv, G, per, n]
        x = x.sub_(top[..., None]).exp_()
        y = y.sub_(top.permute(2, 0, 1, 3)[..., None]).exp_()
        total = x.sum(-1) + y.sum(-1).permute(1, 2, 0, 3)
        o = torch.bmm(x.view(Hkv, -1, S), vp.contiguous()).view(Hkv, G, per, n, D)
        o += torch.bmm(y.view(per * Hkv, G * n, -1), vo.reshape(per * Hkv, -1, D)).view(per, Hkv, G, n, D) \
            .permute(1, 2, 0, 3, 4)
        out[:, :, b0:b1] = o / total[..., None]
    return _packed(out.view(Hkv * G, B, n, D), s["rows"]).to(torch.bfloat16)


def _read(s):
    c = s["case"]
    page, T = c["page"], s["T"]
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = s["kv_len"].long()[seq] - s["cu"].long()[seq + 1] + row
    phys, off = s["table"].long()[seq, pos // page], pos % page
    out = {}
    for name in ("k", "v"):
        x = s[name].view(torch.uint8)[phys, :, off].view(torch.float8_e4m3fn).float()
        out[name] = (x * s[name + "_scale"][phys][..., None]).to(_dtype(c))
    return out


def run(state):
    s = state
    c = s["case"]
    if own:
        import indexer_topk_long_amd as ltk
        if c["op"] == "prompt":
            with torch.no_grad():
                out = ltk.attend_prompt(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], window=c["window"],
                                        return_lse=c["lse"])
            return {"out": out[0], "lse": out[1]} if c["lse"] else {"out": out}
        if c["op"] == "train":
            out = ltk.attend_prompt(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], window=c["window"])
            dq, dk, dv = torch.autograd.grad(out, (s["q"], s["k"], s["v"]), s["dout"])
            return {"out": out.detach(), "dq": dq, "dk": dk, "dv": dv}
        cache = (s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] == "shared":
            return ltk.attend_shared(s["q"], cache, s["table"], s["cu"], s["kv_len"], s["groups"], s["shared_len"])
        k, v = ltk.kv_read(cache, s["table"], s["cu"], s["kv_len"], s["T"], dtype=_dtype(c))
        return {"k": k, "v": v}
    return {"prompt": _prompt, "train": _prompt, "shared": _shared, "read": _read}[c["op"]](s)


# ------------------------------------------------------------- 64 bits

def exact(case, seed):
    """Row blocks of every sequence and head by the definitions, in fp64."""
    s = prepare(case, seed)
    Hkv, D = case["Hkv"], case["D"]
    f64 = dict(device="cuda", dtype=torch.float64)
    if case["op"] == "read":
        page = case["page"]
        out = {}
        for name in ("k", "v"):
            parts = []
            for b, n in enumerate(s["rows"]):
                end = int(s["kv_len"][b])
                pos = torch.arange(end - n, end, device="cuda")
                pg = s["table"][b].long()[pos // page]
                bits = s[name].view(torch.uint8).permute(0, 2, 1, 3)[pg, pos % page].long()
                sign, e, f = 1.0 - 2.0 * (bits >> 7), (bits >> 3) & 15, (bits & 7).double()
                mag = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))
                parts.append(sign * mag * s[name + "_scale"].double()[pg][..., None])
            out[name] = torch.cat(parts)
        return out
    Hq = case["Hq"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    if case["op"] == "shared":
        page, per = case["page"], case["per"]
        out, r0 = torch.zeros(sum(s["rows"]), Hq, D, **f64), 0
        for b, (n, t) in enumerate(zip(s["rows"], s["toks"])):
            key = torch.arange(t, device="cuda")
            pg = s["table"][b].long()[key // page]
            k = s["k"].view(torch.uint8)[pg, :, key % page].view(torch.float8_e4m3fn).double()
            v = s["v"].view(torch.uint8)[pg, :, key % page].view(torch.float8_e4m3fn).double()
            k, v = k * s["k_scale"].double()[pg][..., None], v * s["v_scale"].double()[pg][..., None]
            pos = torch.arange(t - n, t, device="cuda")
            for h in range(Hkv):
                w = s["q"][r0:r0 + n, h * G:(h + 1) * G].double() @ k[:, h].T * scale        # [n, G, t]
                w = torch.softmax(w.masked_fill((key > pos[:, None])[:, None], -math.inf), -1)
                out[r0:r0 + n, h * G:(h + 1) * G] = w @ v[:, h]
            r0 += n
        return out
    pairs = sum(n * m for n, m in zip(s["rows"], s["keys"])) * Hq
    if pairs * (4 if case["op"] == "train" else 1) > 6 * 10 ** 10:   # past about 20 seconds
        return None
    q, k, v = s["q"].detach(), s["k"].detach(), s["v"].detach()
    T, S = q.shape[0], k.shape[0]
    out, lse = torch.zeros(T, Hq, D, **f64), torch.zeros(T, Hq, **f64)
    train = case["op"] == "train"
    if train:
        dq, dk, dv = torch.zeros(T, Hq, D, **f64), torch.zeros(S, Hkv, D, **f64), torch.zeros(S, Hkv, D, **f64)
    r0 = k0 = 0
    for n, m in zip(s["rows"], s["keys"]):
        key = torch.arange(m, device="cuda")
        step = max(1, (1 << 28) // m)
        for x in range(Hq):
            kh, vh = k[k0:k0 + m, x // G].double(), v[k0:k0 + m, x // G].double()
            for i0 in range(0, n, step):
                i1 = min(n, i0 + step)
                r = slice(r0 + i0, r0 + i1)
                pos = torch.arange(m - n + i0, m - n + i1, device="cuda")[:, None]
                see = (key <= pos) & ((key > pos - case["window"]) if case["window"] > 0 else True)
                z = torch.where(see, q[r, x].double() @ kh.T * scale, -math.inf)
                lse[r, x] = torch.logsumexp(z, -1)
                w = torch.exp(z - lse[r, x, None])
                out[r, x] = w @ vh
                if train:
                    g = s["dout"][r, x].double()
                    dz = w * (g @ vh.T - (g * out[r, x]).sum(-1, keepdim=True))
                    dq[r, x] = dz @ kh * scale
                    dk[k0:k0 + m, x // G] += dz.T @ q[r, x].double() * scale
                    dv[k0:k0 + m, x // G] += w.T @ g
        r0, k0 = r0 + n, k0 + m
    if train:
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
