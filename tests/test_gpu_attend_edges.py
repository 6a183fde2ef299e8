"""The paged e4m3 cache's attention where work is cut, joined and planned on
the device: many sequences, many parts of one unit, tables shorter than the
sequences, shared pages, captured calls, and the sparse step as a whole."""
import pytest

from tests.attend_ref import make_batch, make_cache, poison, ref_append, ref_attend, ref_packed
from tests.gpu_util import say
from tests.test_gpu_attend import ATTEND, _attend_case, _dev, _gen, _lists, _within

pytestmark = pytest.mark.gpu


def _widen(table, page, T, Hq, log2_work):
    """The table with room for so many tokens that (row, head) pairs times them pass 2^log2_work: past 2^24 calls of many
    rows take units of 128 rows, past 2^25 of 256."""
    import torch
    more = (2 ** log2_work // (T * Hq) + 1 + page) // page - table.shape[1]
    return torch.nn.functional.pad(table, (0, max(more, 0)), value=-1)


@pytest.mark.parametrize("log2_work", [24, 25])
@pytest.mark.parametrize("case", [c for c in ATTEND if sum(c[0]) * c[3] > 64 * len(c[0])] +
                         [([9, 300], [5000, 300], 2, 16, 64, 64, 0, 0), ([65], [65], 1, 1, 16, 128, 0, 0),
                          ([33, 33], [0, 900], 3, 7, 32, 128, 80, 3), ([400], [100], 1, 2, 16, 64, 0, 0)],
                         ids=lambda c: f"{c[0]}_{c[1]}_h{c[2]}x{c[3]}_p{c[4]}_d{c[5]}_w{c[6]}s{c[7]}")
def test_many_rows_in_large_units(lib, case, log2_work):
    import torch
    rows, lens, Hkv, G, page, D, window, sinks = case
    say("attend", case, log2_work)
    cache, table, cu, n, q = _attend_case(rows, lens, Hkv, G, page, D, 60)
    table = _widen(table, page, sum(rows), Hkv * G, log2_work)
    a = (q.cuda(), _dev(*cache), *_dev(table, cu, n))
    out = lib.attend(*a, window=window, n_sink=sinks)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, window, sinks)
    _within(out, ref, tol, "attend")
    assert torch.equal(out, lib.attend(*a, window=window, n_sink=sinks))


@pytest.mark.parametrize("B,rows,G,Hkv,max_pages", [
    (600, [0, 1, 2], 4, 2, 4),         # few rows a sequence
    (300, [0, 3, 9], 16, 1, 64),       # more than 64 a head: units of 128
    (560, [4, 0, 8, 4, 4], 64, 1, 24),   # 256 a head: units of 256
])
def test_more_sequences_than_one_look(lib, B, rows, G, Hkv, max_pages):
    """Batches whose sequences the kernels look at in several portions, empty ones among them."""
    import torch
    rows = [rows[b % len(rows)] for b in range(B)]
    lens = [r + (7 * b) % 41 for b, r in enumerate(rows)]
    say("sequences", B, sum(rows), G, Hkv)
    g = _gen(61)
    table, cu, n, pages = make_batch(g, rows, lens, 16, max_pages=max_pages)
    cache = make_cache(g, pages, Hkv, 16, 64)
    poison(cache, table, lens, 16)
    q = torch.randn(sum(rows), Hkv * G, 64, generator=g).bfloat16()
    a = (q.cuda(), _dev(*cache), *_dev(table, cu, n))
    out = lib.attend(*a)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 0.125)
    _within(out, ref, tol, f"{B} sequences")
    assert torch.equal(out, lib.attend(*a))
    idx = _lists(_gen(62), rows, lens, 20)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, 0.125, idx=idx)
    _within(lib.attend_selected(*a, idx.cuda()), ref, tol, f"{B} sequences, selected")


@pytest.mark.parametrize("T,L,G,D,window,sinks", [
    (1, 20000, 4, 64, 0, 0), (1, 20000, 20, 128, 0, 0), (20, 20000, 8, 64, 0, 0), (70, 9000, 4, 128, 0, 0),
    (130, 20000, 8, 64, 0, 0), (110, 20000, 16, 128, 0, 0),   # units of 128 rows, of 256
    (40, 9000, 8, 128, 5000, 33), (1, 20000, 3, 128, 9000, 7),
])
def test_one_unit_in_many_parts(lib, T, L, G, D, window, sinks):
    import torch
    say("parts", T, L, G, D, window, sinks)
    cache, table, cu, n, q = _attend_case([T], [L], 1, G, 64, D, 63)
    a = (q.cuda(), _dev(*cache), *_dev(table, cu, n))
    out = lib.attend(*a, window=window, n_sink=sinks)
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5, window, sinks)
    _within(out, ref, tol, "parts")
    assert torch.equal(out, lib.attend(*a, window=window, n_sink=sinks))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [576, 4096, 16384])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5), (3, 70)])
def test_chunks_over_holes_and_short_tables(lib, D, cap, window, sinks):
    """Many rows: pages missing in the middle, tokens past the table or a table far wider than the tokens (units of 32,
    of 128 and of 256 rows), freed pages before the window, rows before cu[0] and behind cu[B]."""
    import torch
    page, Hkv, G = 16, 2, 8
    rows, lens = [260, 0, 77], [700, 5, 500]
    g = _gen(64)
    table, cu, n, pages = make_batch(g, rows, lens, page, max_pages=cap // page)
    table[0, 7], table[0, 20:22], table[2, 3] = -1, torch.tensor([pages, 2 ** 31 - 1]).int(), -2 ** 31
    if window:
        table[0, 5:15] = -5              # positions 80 .. 239: behind every row's window (and the sinks)
    cache = make_cache(g, pages, Hkv, page, D)
    poison(cache, table, lens, page)
    T = sum(rows) + 5
    q = torch.randn(T, Hkv * G, D, generator=g).bfloat16()
    cu = cu + 2
    out = torch.full((T, Hkv * G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    say("chunk", D, cap, window, sinks)
    lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n), window=window, n_sink=sinks, out=out)
    ref, tol, written = ref_attend(q, cache, table, cu, n, D ** -0.5, window, sinks)
    assert bool((out.cpu()[~written] == 9).all()) and int(written.sum()) == 337
    _within(out.cpu()[written], ref[written], tol[written], "chunk")


def test_scales_and_sharp_softmax_of_chunks(lib):
    """Many rows with scales that are no powers of two, scores in the hundreds, and value scales far apart."""
    import torch
    for D, pow2, qs in ((64, False, 60.0), (128, True, 40.0)):
        cache, table, cu, n, q = _attend_case([150], [400], 2, 4, 16, D, 65, pow2, qs)
        cache[3][table[0].long()] *= torch.exp2(torch.linspace(-40, 40, 25).round())[:, None]
        for t in (table, _widen(table, 16, 150, 8, 24), _widen(table, 16, 150, 8, 25)):
            out = lib.attend(q.cuda(), _dev(*cache), *_dev(t, cu, n), window=300, n_sink=2)
            ref, tol, _ = ref_attend(q, cache, t, cu, n, D ** -0.5, 300, 2)
            _within(out, ref, tol, f"D {D}")


def test_shared_pages_and_equal_sequences(lib):
    """Two sequences that share their first pages, and two that are the same."""
    import torch
    page, D, Hkv, G = 32, 128, 2, 4
    g = _gen(66)
    table, cu, n, pages = make_batch(g, [3, 90, 90], [200, 190, 190], page)
    table[1, :3] = table[0, :3]
    table[2] = table[1]
    cache = make_cache(g, pages, Hkv, page, D)
    q = torch.randn(183, Hkv * G, D, generator=g).bfloat16()
    q[93:] = q[3:93]
    out = lib.attend(q.cuda(), _dev(*cache), *_dev(table, cu, n))
    ref, tol, _ = ref_attend(q, cache, table, cu, n, D ** -0.5)
    _within(out, ref, tol, "shared")


def test_one_workspace_for_calls_of_many_kinds(lib):
    """A workspace used by calls of other kinds and sizes before, on one stream, as it is left."""
    import torch
    import indexer_topk_long_amd as ltk
    g = _gen(67)
    cases = [([1], [9000], 1, 4, 64, 128), ([200], [900], 2, 8, 64, 128), ([1, 1], [50, 3000], 2, 2, 64, 64),
             ([300], [300], 1, 8, 64, 64)]
    built = [_attend_case(*c, seed=68 + i) for i, c in enumerate(cases)]
    built = [(c, _widen(t, 64, q.shape[0], q.shape[1], 24 + i % 2) if i in (1, 3) else t, cu, n, q)
             for i, (c, t, cu, n, q) in enumerate(built)]
    need = max(ltk.attend_workspace_bytes(0, q.shape[0], q.shape[1], c[0].shape[1], q.shape[2], table.shape[0],
                                          table.shape[1] * 64) for c, table, cu, n, q in built)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    args = [(q.cuda(), _dev(*c), *_dev(t, cu, n)) for c, t, cu, n, q in built]
    want = [lib.attend(*a) for a in args]
    graphs = []
    for a in args:      # captured over the same workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o = lib.attend(*a, workspace=ws)
        graphs.append((gr, o))
    for turn in range(3):
        for i in (0, 1, 2, 3, 1, 0, 3, 2):
            assert torch.equal(lib.attend(*args[i], workspace=ws), want[i]), (turn, i)
            graphs[i][1].zero_()
            graphs[i][0].replay()
            assert torch.equal(graphs[i][1], want[i]), (turn, i)


def test_chunk_and_packed_captured_and_replayed(lib):
    """Lengths, rows' starts, lists and their lengths change in place between replays."""
    import torch
    g = _gen(69)
    page, D, Hkv, G, T, group, cap = 16, 64, 2, 8, 64, 16, 300
    table, _, _, pages = make_batch(g, [T], [900], page)
    table = _widen(table, page, T, Hkv * G, 24)
    cache = make_cache(g, pages, Hkv, page, D)
    dc, dt = _dev(*cache), table.cuda()
    q = torch.randn(T, Hkv * G, D, generator=g).bfloat16().cuda()
    cu, n = torch.tensor([0, T]).int().cuda(), torch.tensor([T]).int().cuda()
    shared = torch.zeros(4, cap, dtype=torch.int32, device="cuda")
    masks, lens = torch.zeros_like(shared).view(torch.uint32), torch.zeros(4, dtype=torch.int32, device="cuda")
    run = lambda: (lib.attend(q, dc, dt, cu, n, window=200, n_sink=3), lib.attend(q, dc, dt, cu, n),
                   lib.attend_packed(q, dc, dt, n, shared, masks, lens, group))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i, L in enumerate((64, 900, 333, 10, 512)):
        n.fill_(L)
        cu.copy_(torch.tensor([i, T - i]).int())
        shared.copy_(torch.stack([torch.randperm(900, generator=g)[:cap] for _ in range(4)]).int())
        masks.view(torch.int32).copy_(torch.randint(0, 1 << 16, (4, cap), generator=g).int())
        lens.copy_(torch.tensor([cap, 0, 1, 37 * i]).int())
        for o in outs:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = run()
        torch.cuda.synchronize()
        for o, w, sl in zip(got, want, (slice(i, T - i), slice(i, T - i), slice(0, T))):
            assert torch.equal(o[sl], w[sl]), i
        ref, tol, written = ref_attend(q.cpu(), cache, table, cu.cpu(), n.cpu(), 0.125)
        _within(got[1].cpu()[written], ref[written], tol[written], f"length {L}")
        ref, tol = ref_packed(q.cpu(), cache, table, n.cpu(), shared.cpu(), masks.cpu(), lens.cpu(), group, 0.125)
        _within(got[2], ref, tol, f"packed, length {L}")


@pytest.mark.parametrize("G,group,D", [(1, 32, 64), (5, 7, 128), (4, 24, 64), (7, 14, 128), (12, 9, 64), (16, 8, 128),
                                       (3, 32, 128), (40, 2, 64)])
def test_packed_groups_over_odd_lists(lib, G, group, D):
    """Groups of few and of many (row, head) pairs, the last one not full: holes in the table, keys after some rows of a
    group, repeated entries, lengths past cap, bits of rows that are not there, rows that select nothing, long lists."""
    import torch
    T, L, cap = 3 * group - 1, 2600, 2500
    cache, table, cu, n, q = _attend_case([T], [L], 2, G, 16, D, 71)
    table[0, 4], table[0, 100] = -1, 2 ** 31 - 1
    poison(cache, torch.where(table == 2 ** 31 - 1, -1, table), [L], 16)
    g = _gen(72)
    shared = torch.stack([torch.randperm(L + 20, generator=g)[:cap] for _ in range(3)]).int()
    shared[:, 5], shared[1, 9], shared[2, 11] = -3, 2 ** 31 - 1, shared[2, 10]
    shared[:, 40:40 + T // 2] = torch.arange(L - T, L - T + T // 2).int()      # the rows themselves
    masks = torch.randint(0, 1 << 32, (3, cap), generator=g)
    masks[0] &= ~1                                  # the first row selects nothing
    masks = masks.to(torch.uint32)
    lens = torch.tensor([cap + 50, 33, cap]).int()
    a = (q.cuda(), _dev(*cache), *_dev(table, n, shared, masks, lens), group)
    say("packed", G, group, D)
    out = lib.attend_packed(*a)
    ref, tol = ref_packed(q, cache, table, n, shared, masks, lens, group, D ** -0.5)
    assert bool((out[0] == 0).all())
    _within(out, ref, tol, "odd lists")
    assert torch.equal(out, lib.attend_packed(*a))


@pytest.mark.parametrize("T,Hkv,topk", [(0, 2, 40), (1, 2, 40), (9, 1, 64), (520, 4, 100), (700, 2, 33)])
def test_sparse_step(lib, T, Hkv, topk):
    """Append, select and attend in one call, on a stream of its own: few rows on their own lists, long chunks packed."""
    import torch
    import indexer_topk_long_amd as ltk
    g = _gen(70)
    page, D, G, L, H = 32, 64, 2, 900, 4
    table, cu, n, pages = make_batch(g, [T], [L], page)
    cache = make_cache(g, pages, Hkv, page, D)
    k, v = (torch.randn(T, Hkv, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(T, Hkv * G, D, generator=g).bfloat16()
    f = 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    iq, ik = torch.randn(T, H, D, generator=g).bfloat16(), torch.randn(L, D, generator=g).bfloat16()
    w = torch.rand(T, H, generator=g)
    want = ref_append(k, v, cache, table, cu, n, f, False)
    dc = _dev(*cache)
    dev = _dev(q, k, v, table, n, iq, ik, w, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, idx = ltk.sparse_step(dev[0], dev[1], dev[2], dc, dev[3], dev[4], dev[5], dev[6], dev[7], topk, inv_freq=dev[8])
    side.synchronize()
    assert out.shape == q.shape and idx.shape == (T, topk)
    for a, b in zip(dc, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))
    if T == 0:
        return
    pos = torch.arange(L - T, L, dtype=torch.int32, device="cuda")
    assert torch.equal(idx.sort(1)[0], ltk.score_select(dev[5], dev[6], dev[7], pos, topk).sort(1)[0])
    qr = lib.kv_append(dev[1], dev[2], dc, dev[3], *_dev(cu, n, f), q=dev[0]).cpu()   # the same rows again: the same cache
    ref, tol, _ = ref_attend(qr, want, table, cu, n, D ** -0.5, idx=idx.cpu())
    _within(out, ref, tol, f"{T} rows")


@pytest.mark.parametrize("G,group", [(8, 16), (2, 8)])
def test_one_workspace_sized_for_the_largest_call(lib, G, group):
    """A buffer of what the size function gives for the longest batch serves the short steps too, of every kind."""
    import torch
    import indexer_topk_long_amd as ltk
    g = _gen(73)
    L, T, Hkv, D, topk = 1500, 600, 4, 64, 700
    cache, table, cu, n, q = _attend_case([T], [L], Hkv, G, 16, D, 74)
    dc, dt, dn = _dev(*cache), table.cuda(), n.cuda()
    idx = torch.stack([torch.randperm(L - T + 1, generator=g)[:topk] for _ in range(T)]).int().cuda()
    sh, m, ln = ltk.dsa_pack(idx, L, group)
    sizes = [ltk.attend_workspace_bytes(k, T, Hkv * G, Hkv, D, 1, e, gr)
             for k, e, gr in ((0, table.shape[1] * 16, 0), (1, topk, 0), (2, group * topk, group))]
    for t in (T, 1, 33, 3, 130, T):
        r = slice(0, t)      # the first rows, as the sequence's last tokens
        qt, ng = q[r].contiguous().cuda(), -(-t // group)
        c = torch.tensor([0, t]).int().cuda()
        calls = (lambda **k: ltk.attend(qt, dc, dt, c, dn, **k), lambda **k: ltk.attend_selected(qt, dc, dt, c, dn, idx[r], **k),
                 lambda **k: ltk.attend_packed(qt, dc, dt, dn, sh[:ng], m[:ng], ln[:ng], group, **k))
        for call, size in zip(calls, sizes):
            ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
            assert torch.equal(call(workspace=ws), call()), t


@pytest.mark.parametrize("T,G,log2_work", [(3, 4, 0), (80, 4, 0), (80, 4, 24), (140, 4, 25)])
@pytest.mark.parametrize("seqs", [1, 3, 600])
def test_batches_whose_sequences_have_no_rows(lib, T, G, log2_work, seqs):
    """Rows that belong to no sequence, as a captured step has them when its batch is empty: nothing is written; in the
    next call over the same workspace they have sequences again."""
    import torch
    import indexer_topk_long_amd as ltk
    say("no rows", T, G, log2_work, seqs)
    Hkv, D = 2, 64
    if log2_work:
        T *= seqs                # (row, head) pairs for the many-row kernels
    cache, table, cu, n, q = _attend_case([T] + [0] * (seqs - 1), [T + 200] + [90] * (seqs - 1), Hkv, G, 16, D, 76)
    if log2_work:
        table = _widen(table, 16, T, Hkv * G, log2_work)
    dc, (dt, dcu, dn) = _dev(*cache), _dev(table, cu, n)
    idx = torch.zeros(T, 7, dtype=torch.int32, device="cuda")
    k = torch.ones(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    need = ltk.attend_workspace_bytes(0, T, Hkv * G, Hkv, D, seqs, table.shape[1] * 16)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    want = lib.attend(q.cuda(), dc, dt, dcu, dn)
    before = [t.clone() for t in dc]
    for at in (0, T):
        none = torch.full_like(dcu, at)
        out = torch.full_like(q, 5.0).cuda()
        lib.attend(q.cuda(), dc, dt, none, dn, out=out, workspace=ws)
        lib.attend_selected(q.cuda(), dc, dt, none, dn, idx, out=out)
        assert lib.kv_append(k, k, dc, dt, none, dn, None, q.cuda(), q_out=out) is out
        assert bool((out == 5).all()), at
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, dc))
        assert torch.equal(lib.attend(q.cuda(), dc, dt, dcu, dn, workspace=ws), want)
