"""One sparse-attention step of a sequence: the new tokens' keys and values go
to the paged cache, the indexer selects each row's keys, and the rows attend
to their selections -- a decode or speculative-decode step, or a prefill chunk
(the LiteTopK pages, arXiv abstract: neighbouring rows of a chunk attend
jointly to one packed list)."""
from __future__ import annotations

import math

from ._binding import Opts, _expect, dsa_pack, score_select
from .attention import attend_packed, attend_selected, kv_append

# Packing pays where several key/value heads read each list: from this many
# heads, and rows times heads, the selections are packed in groups of
# PACK_GROUP rows.  (topk 2,048, eight heads: 256 rows take 139 us on their own
# lists, 49 us to pack and 78 us packed; four heads, 1,024 rows: 266 us against
# 53 + 133; two heads, 2,048 rows: 273 us against 55 + 225.)
PACK_HEADS, PACK_WORK, PACK_GROUP = 4, 2048, 16


def sparse_step(q, k, v, cache, page_table, kv_len, index_q, index_k, index_w, topk: int, inv_freq=None,
                interleaved: bool = False, scale=None, sample=None, index_q_scale=None, index_k_scale=None,
                opts: Opts | None = None, out=None):
    """Appends the last T tokens of one sequence and attends from them.

    q [T, Hq, D], k and v [T, Hkv, D] bfloat16, cache, page_table [1,
    max_pages] and kv_len [1] (the new tokens included) as for kv_append;
    inv_freq and interleaved rotate q and k.  index_q [T, H, Di], index_w
    [T, H] and index_k [L, Di] are score_select's q, w and k (and their scales
    and sample): index_k holds the index keys of the sequence's tokens, the new
    ones included, so L is the sequence's length.

    Returns (out [T, Hq, D] bfloat16, idx [T, topk] int32): idx is the next
    step's sample.  Long chunks attend in groups of PACK_GROUP rows to
    their packed selections (the same result, but for the order of the sums)
    where dsa_pack takes them: PACK_GROUP * topk <= 32768 and L <= 2^26.

    Tensors are on one device; the step runs on that device's current stream.
    A refused call leaves the cache as it was: the append is the last step that
    can be refused.
    """
    import torch
    if out is not None:
        _expect(out.shape == q.shape and out.dtype == torch.bfloat16 and out.device == q.device and out.is_contiguous(),
                f"out must be a contiguous bfloat16 tensor {tuple(q.shape)} on {q.device}")
    if scale is not None:   # finite, also times log2(e) in fp32
        _expect(abs(scale) * math.log2(math.e) <= torch.finfo(torch.float32).max, f"scale {scale} is out of range")
    with torch.cuda.device_of(q):   # the selection runs on the current device's stream
        T, L, Hkv = q.shape[0], index_k.shape[0], k.shape[1]
        at = torch.arange(T + 1, dtype=torch.int32, device=q.device)
        cu = at[::max(T, 1)][:2].contiguous() if T else at.expand(2).contiguous()
        pos = kv_len - T + at[:T]
        idx = score_select(index_q, index_k, index_w, pos, topk, sample=sample, q_scale=index_q_scale,
                           k_scale=index_k_scale, opts=opts)
        packed = Hkv >= PACK_HEADS and T * Hkv >= PACK_WORK and PACK_GROUP * topk <= 32768 and L <= 1 << 26
        if packed:
            shared, masks, lens = dsa_pack(idx, L, PACK_GROUP)
        qr = kv_append(k, v, cache, page_table, cu, kv_len, inv_freq, q=q, interleaved=interleaved)
        if packed:
            return attend_packed(qr, cache, page_table, kv_len, shared, masks, lens, PACK_GROUP, scale, out), idx
        return attend_selected(qr, cache, page_table, cu, kv_len, idx, scale, out), idx
