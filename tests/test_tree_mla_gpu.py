"""Latent attention of drafted token trees over the paged cache (idx_tree_mla)
against float64, element by element within the bound of tests/paged_helpers.py."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, Paged, bf, check_tree, mask_dev, random_tree

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _run(X, paged, q, cnts, n, mask=None, indices=None, scale=SCALE, dtype=torch.bfloat16, given=True, **kw):
    B, _, H = q.shape[:3]
    out = torch.full((B, n, H, LAT), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((B, n, H), 5.0, dtype=torch.float32, device="cuda")
    X.tree_mla(q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), scale,
               max_len=max(max(paged.lens), 1), counts=dev(np.array(cnts, np.int32)) if given else None,
               tree_mask=mask_dev(mask) if mask is not None else None,
               indices=dev(indices) if indices is not None else None, out=out, lse=lse, **kw)
    assert X.status() == (0, 0)
    return out, lse


@pytest.mark.parametrize("n,H,page,ctxs,cnts,tree", [
    (1, 16, 64, [0, 1, 126, 127, 128, 255], None, False),        # one token; lengths around a 128-key tile
    (1, 1, 1, [0, 130, 300], None, False),                       # one head, pages of one row
    (1, 128, 64, [1000, 3, 517], None, False),                   # all heads
    (2, 5, 33, [500, 0, 257], [2, 1, 2], True),                  # odd heads; pages end inside a tile
    (7, 16, 48, [0, 129, 900], [7, 3, 0], True),                 # a sequence without rows
    (13, 20, 16, [1, 640], [13, 6], True),                       # 260 rows: row groups cross tokens
    (64, 8, 100, [70, 0], [64, 33], True),                       # the widest mask
    (4, 128, 128, [383, 128], [4, 4], True),
    (3, 256, 200, [450], None, False),                           # more heads than one block of 128
    (1, 16, 64, [20000], None, False),                           # one long sequence, split over the GPU
    (5, 24, 16, [9000, 17, 4000, 0, 2500], [5, 5, 1, 2, 4], True),
])
def test_dense_matches_float64(n, H, page, ctxs, cnts, tree):
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(n * 1000 + H)
    B = len(ctxs)
    real = cnts or [n] * B
    paged = Paged(rng, [a + m for a, m in zip(ctxs, real)], page).fill(rng)
    q64, q = bf(rng.standard_normal((B, n, H, DIM)))
    mask = [random_tree(rng, n) for _ in range(B)] if tree else None
    if tree and n > 1:
        mask[0][n - 1] = 0                                       # a row that sees no draft
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = _run(X, paged, q, real, n, mask, dtype=dtype, given=cnts is not None)
        check_tree(out, lse, q64, paged, real, SCALE, mask, untouched=5.0)


@pytest.mark.parametrize("n,H,page,ctxs,cnts,k,tree", [
    (1, 16, 64, [5000, 300, 0], None, 256, False),               # a selection wider than a context
    (1, 128, 64, [3000, 2500], None, 2048, False),
    (2, 64, 33, [700, 1], [2, 1], 100, True),
    (7, 16, 48, [2000, 0, 90], [7, 7, 0], 130, True),
    (3, 5, 16, [1000, 129], None, 1, False),                     # one selected position
    (16, 1, 100, [513, 77], [16, 9], 127, True),
    (2, 200, 64, [800], None, 128, False),
])
def test_selected_matches_float64(n, H, page, ctxs, cnts, k, tree):
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(n * 1000 + H + k)
    B = len(ctxs)
    real = cnts or [n] * B
    paged = Paged(rng, [a + m for a, m in zip(ctxs, real)], page).fill(rng)
    q64, q = bf(rng.standard_normal((B, n, H, DIM)))
    mask = [random_tree(rng, n) for _ in range(B)] if tree else None
    idx = np.full((B, n, k), -1, np.int32)
    for b in range(B):
        for i in range(n):
            m = min(k, ctxs[b])
            idx[b, i, :m] = rng.choice(ctxs[b], m, replace=False) if m else 0
            rng.shuffle(idx[b, i])                               # −1 anywhere in the row
    if k > 8 and ctxs[0] > 20:
        idx[0, 0, :3] = idx[0, 0, 3]                             # one position four times: it counts four times
        idx[0, 0, 4] = ctxs[0]                                   # a draft's slot, past the end, below zero: nothing
        idx[0, 0, 5] = ctxs[0] + real[0] + 1000
        idx[0, 0, 6] = -2147483648
    out, lse = _run(X, paged, q, real, n, mask, idx, given=cnts is not None)
    check_tree(out, lse, q64, paged, real, SCALE, mask, idx, untouched=5.0)


@pytest.mark.parametrize("scale", [3.0, -0.2, 0.0, 1e-3])
def test_scales(scale):
    """A peaky softmax (the reference maximum rises again and again), a negative
    scale, none, a flat one."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(5)
    paged = Paged(rng, [1500, 40], 64).fill(rng)
    t = np.arange(1500)                                          # scores that grow along the sequence
    for b in range(2):
        for i in range(paged.lens[b]):
            pg = paged.table[b, i // 64]
            paged.cache[pg, i % 64], _ = bf(paged.cache[pg, i % 64] * (0.2 + 0.8 * i / 1500))
    q64, q = bf(rng.standard_normal((2, 3, 16, DIM)))
    out, lse = _run(X, paged, q, [3, 3], 3, scale=scale)
    check_tree(out, lse, q64, paged, [3, 3], scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H,n", [(16, 4), (128, 3)])
def test_numbers_in_masked_places_reach_no_other_row(bad, H, n):
    """A draft's cache row that is not finite: rows that do not see it are as if
    it were not there, rows that see it are not finite.  Unheld rows are NaN in
    every test of this file."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(6)
    ctx = 130
    paged = Paged(rng, [ctx + n], 64).fill(rng)
    mask = [[1 << i for i in range(n)]]                          # every draft sees itself alone
    t = ctx + 1
    paged.cache[paged.table[0, t // 64], t % 64, :] = bad        # draft 1
    q64, q = bf(rng.standard_normal((1, n, H, DIM)))
    for idx in (None, np.arange(60, dtype=np.int32)[None, None].repeat(n, 1)):
        out, lse = _run(X, paged, q, [n], n, mask, idx)
        assert not torch.isfinite(out[0, 1]).all(dim=-1).any()
        keep = [i for i in range(n) if i != 1]
        good = Paged.__new__(Paged)
        good.__dict__.update(paged.__dict__)
        good.cache = paged.cache.copy()
        good.cache[paged.table[0, t // 64], t % 64, :] = 0.0
        q64k = q64[:, keep]
        # rows 0, 2, 3 … see the context and themselves
        from tests.paged_helpers import UB, row_positions, tree_row
        for i in keep:
            pos = row_positions(good.lens, [n], mask, idx, 0, i)
            o, ls, bound, lerr = tree_row(q64[0, i], good.rows(0, ctx + n)[pos], SCALE)
            assert np.all(np.abs(out[0, i].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB) + 1e-30)
            assert np.all(np.abs(lse[0, i].double().cpu().numpy() - ls) <= lerr)


def test_scores_that_are_infinite_or_huge():
    """A context row of the type's largest values: its score is +inf or −inf in
    fp32 terms or huge; heads where it is hugely negative ignore it."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(7)
    paged = Paged(rng, [200], 64).fill(rng)
    big = 3.3e38
    paged.cache[paged.table[0, 1], 5, :], _ = bf(np.full(DIM, big))
    q64, q = bf(-np.abs(rng.standard_normal((1, 1, 16, DIM))))  # scores with the big row: −inf
    out, lse = _run(X, paged, q, [1], 1)
    assert torch.isfinite(lse).all() and torch.isfinite(out).all()
    kv = np.delete(paged.rows(0, 200), 64 + 5, axis=0)
    from tests.paged_helpers import tree_row, UB
    o, ls, bound, lerr = tree_row(q64[0, 0], kv, SCALE)
    assert np.all(np.abs(out[0, 0].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB))
    assert np.all(np.abs(lse[0, 0].double().cpu().numpy() - ls) <= lerr)


def test_errors_that_depend_on_data():
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(8)
    paged = Paged(rng, [300, 300, 300], 64).fill(rng)
    q64, q = bf(rng.standard_normal((3, 2, 16, DIM)))

    def go(lens, cnts, table=None, max_len=300):
        out = torch.full((3, 2, 16, LAT), 5.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((3, 2, 16), 5.0, device="cuda")
        X.tree_mla(q.cuda(), paged.cache_dev(), paged.table_dev() if table is None else dev(table),
                   dev(np.array(lens, np.int32)), SCALE, max_len=max_len, counts=dev(np.array(cnts, np.int32)), out=out,
                   lse=lse)
        return out, lse, X.status()

    for lens, cnts in (([301, 300, 300], [2, 2, 2]), ([1, 300, 300], [2, 2, 2]), ([300, 300, 300], [3, 2, 2]),
                       ([300, 300, 300], [-1, 2, 2])):
        out, lse, st = go(lens, cnts)
        assert st == (-7, X.DEV_ERR_LENGTH)
        assert (out[0] == 5).all() and (lse[0] == 5).all()       # the bad sequence's outputs are as they were
        check_tree(out[1:], lse[1:], q64[1:], _tail(paged), [2, 2], SCALE)
    table = paged.table.copy()
    table[0, 1] = paged.num_pages                                # a page that is none: its 64 positions are not seen
    table[1, 2] = -5
    out, lse, st = go([300] * 3, [2] * 3, table)
    assert st == (-7, X.DEV_ERR_PAGE)
    from tests.paged_helpers import UB, tree_row
    for b, gone in ((0, 1), (1, 2), (2, None)):
        for i in range(2):
            pos = [t for t in range(298 + i + 1) if t // 64 != gone]
            o, ls, bound, lerr = tree_row(q64[b, i], paged.rows(b, 300)[pos], SCALE)
            assert np.all(np.abs(out[b, i].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB))
            assert np.all(np.abs(lse[b, i].double().cpu().numpy() - ls) <= lerr)


def _tail(paged):
    t = Paged.__new__(Paged)
    t.__dict__.update(paged.__dict__)
    t.table, t.lens = paged.table[1:], paged.lens[1:]
    return t


def test_streams_graphs_and_repeated_calls_agree():
    """The same bits on another stream, from two captured graphs with workspaces
    of their own replayed at once, after the inputs changed in place, and from a
    workspace that held another call's results."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(9)
    B, n, H = 6, 3, 16
    lens = [4000, 129, 900, 3, 7000, 2500]
    paged = Paged(rng, lens, 64).fill(rng)
    _, q = bf(rng.standard_normal((B, n, H, DIM)))
    qd, cache, table, L = q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(lens, np.int32))
    call = lambda **kw: X.tree_mla(qd, cache, table, L, SCALE, max_len=7000, **kw)
    want, wl = call()
    again, al = call()
    assert torch.equal(want, again) and torch.equal(wl, al)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, l2 = call(stream=s)
    s.synchronize()
    assert torch.equal(want, o2) and torch.equal(wl, l2)
    graphs = []
    for _ in range(2):
        o = torch.zeros_like(want)
        ws = torch.full((max(16, X.tree_mla_workspace_size(B, n, H, 7000)),), 0xFF, dtype=torch.uint8, device="cuda")
        lse = torch.zeros_like(wl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out=o, lse=lse, ws=ws)
        graphs.append((g, o, lse, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for r in range(3):
        for (g, o, lse, ws), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for g, o, lse, ws in graphs:
        assert torch.equal(o, want) and torch.equal(lse, wl)
    qd.copy_(-qd)
    want2, _ = call()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][1], want2) and not torch.equal(want, want2)
    assert X.status() == (0, 0)


@pytest.mark.parametrize("n,H,page,ctxs,cnts,k,tree", [
    (1, 24, 64, [127, 128, 1000], None, 0, False),               # 17 to 32 rows per key set
    (2, 16, 48, [0, 385, 64], [2, 1, 2], 0, True),
    (2, 10, 16, [600, 100], None, 130, True),
    (1, 64, 64, [3000, 1, 255], None, 0, False),                 # 33 to 64 rows
    (4, 16, 33, [1000, 257], [4, 3], 0, True),
    (1, 40, 100, [900], None, 300, False),
    (1, 65, 64, [400, 63], None, 0, False),                      # one row more than the narrow kernels hold
    (9, 16, 64, [700, 0], [9, 8], 0, True),                      # a second group of 128 rows for one sequence only
    (1, 128, 64, [20000], None, 0, False),                       # one long sequence over the whole GPU, all heads
    (2, 128, 16, [6000, 6001], None, 4000, True),                # many pieces of a selection
])
def test_row_counts_of_every_kernel(n, H, page, ctxs, cnts, k, tree):
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(n * 1000 + H + k + 1)
    B = len(ctxs)
    real = cnts or [n] * B
    paged = Paged(rng, [a + m for a, m in zip(ctxs, real)], page).fill(rng)
    q64, q = bf(rng.standard_normal((B, n, H, DIM)))
    mask = [random_tree(rng, n) for _ in range(B)] if tree else None
    idx = None
    if k:
        idx = np.full((B, n, k), -1, np.int32)
        for b in range(B):
            for i in range(n):
                m = min(k, ctxs[b])
                idx[b, i, :m] = rng.choice(ctxs[b], m, replace=False)
    out, lse = _run(X, paged, q, real, n, mask, idx, given=cnts is not None)
    check_tree(out, lse, q64, paged, real, SCALE, mask, idx, untouched=5.0)


@pytest.mark.parametrize("H", [3, 20, 64, 100, 200])
@pytest.mark.parametrize("ctxs", [[6000, 130, 1300, 0, 9000], [12000], [700, 900, 800], [256, 257]])
def test_items_of_few_and_many_pieces(H, ctxs):
    """Contexts cut into one piece, a few, or one for most SMs, side by side; the
    join's order is fixed, so two calls give the same bits."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(H + len(ctxs))
    B = len(ctxs)
    paged = Paged(rng, [c + 1 for c in ctxs], 64).fill(rng)
    q64, q = bf(rng.standard_normal((B, 1, H, DIM)))
    for dtype in (torch.bfloat16, torch.float32):
        out, lse = _run(X, paged, q, [1] * B, 1, dtype=dtype)
        check_tree(out, lse, q64, paged, [1] * B, SCALE)
        again, lse2 = _run(X, paged, q, [1] * B, 1, dtype=dtype)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("B,n,H,ctx,k", [
    (1, 1, 16, 300, 0), (1, 1, 3, 129, 0), (2, 3, 20, 700, 0), (1, 2, 64, 2000, 0), (1, 1, 128, 5000, 0),
    (3, 4, 128, 400, 0), (1, 2, 16, 900, 300), (2, 5, 128, 900, 260), (60, 1, 16, 500, 0), (1, 1, 16, 40000, 0),
])
def test_workspace_of_exactly_the_stated_size(B, n, H, ctx, k):
    """The call needs no byte more than it says, and writes none behind."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(B * 100 + H)
    paged = Paged(rng, [max(n, ctx - 37 * b) + n for b in range(B)], 64).fill(rng)
    q64, q = bf(rng.standard_normal((B, n, H, DIM)))
    idx = None
    if k:
        idx = np.stack([[rng.choice(paged.lens[b] - n, k, replace=False) for _ in range(n)] for b in range(B)]).astype(np.int32)
    need = X.tree_mla_workspace_size(B, n, H, max(paged.lens), k)
    assert (need > 0) == ((k + n if k else max(paged.lens)) > 256)    # up to 256 keys stay whole
    room = torch.full((need + 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = _run(X, paged, q, [n] * B, n, indices=idx, given=False, ws=room[:need])
    assert bool((room[need:] == 0xA5).all())
    check_tree(out, lse, q64, paged, [n] * B, SCALE, None, idx)
    if need:
        with pytest.raises(X.IdxError):
            _run(X, paged, q, [n] * B, n, indices=idx, given=False, ws=room[:need - 16])


@pytest.mark.parametrize("H", [4, 30, 128])
@pytest.mark.parametrize("scale", [3.0, -0.3])
def test_reference_maximum_rises_in_every_kernel(H, scale):
    """Scores that grow along a sequence cut into pieces, with peaky softmaxes."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(11)
    L = 2500
    paged = Paged(rng, [L, 700], 64).fill(rng)
    for b in range(2):
        for i in range(paged.lens[b]):
            pg = paged.table[b, i // 64]
            paged.cache[pg, i % 64], _ = bf(paged.cache[pg, i % 64] * (0.1 + 0.9 * i / L))
    q64, q = bf(rng.standard_normal((2, 1, H, DIM)))
    out, lse = _run(X, paged, q, [1, 1], 1, scale=scale)
    check_tree(out, lse, q64, paged, [1, 1], scale)


def test_large_batch_of_short_sequences_and_empty_batches():
    """More sequences than a CTA has threads, without rows or a context here and
    there; then a batch in which no sequence has a row."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(12)
    B, n, H = 1300, 2, 3
    cnts = [int(x) for x in rng.integers(0, 3, B)]
    lens = [c + int(rng.integers(0, 40)) for c in cnts]
    paged = Paged(rng, lens, 16).fill(rng)
    q64, q = bf(rng.standard_normal((B, n, H, DIM)))
    out, lse = _run(X, paged, q, cnts, n)
    check_tree(out, lse, q64, paged, cnts, SCALE, untouched=5.0)
    none = [0] * B
    out, lse = _run(X, paged, q, none, n)
    assert (out == 5).all() and (lse == 5).all()


def test_pages_past_four_gigabytes():
    """Cache rows whose byte offsets pass 32 bits, appended and attended to."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(13)
    pages, page, H, L = 62000, 64, 16, 200
    cache = torch.zeros((pages, page, DIM), dtype=torch.bfloat16, device="cuda")      # 4.6 GB
    table = np.array([[pages - 1, pages - 3, 59000, pages - 2]], np.int32)
    kv64, kv = bf(rng.standard_normal((1, L, DIM)))
    gain, cos, sin = np.ones(LAT, np.float32), np.ones((1, L, 32), np.float32), np.zeros((1, L, 32), np.float32)
    X.latent_append(kv.cuda(), dev(gain), 0.0, dev(cos), dev(sin), dev(np.zeros(1, np.int32)), dev(table), cache)
    t = np.arange(L)
    rows = cache[torch.from_numpy(table[0, t // page]).long().cuda(), torch.from_numpy(t % page).cuda()]
    rms = np.sqrt(np.mean(kv64[0, :, :LAT] ** 2, axis=1, keepdims=True))
    got = rows.double().cpu().numpy()
    assert np.all(np.abs(got[:, :LAT] - kv64[0, :, :LAT] / rms) <= np.abs(kv64[0, :, :LAT] / rms) * (2 ** -8 + 2 ** -15))
    q64, q = bf(rng.standard_normal((1, 1, H, DIM)))
    for idx in (None, rng.choice(L - 1, 64, replace=False).astype(np.int32)[None, None]):
        out, lse = X.tree_mla(q.cuda(), cache, dev(table), dev(np.array([L], np.int32)), SCALE, max_len=L,
                              indices=None if idx is None else dev(idx))
        assert X.status() == (0, 0)
        from tests.paged_helpers import UB, tree_row
        pos = list(range(L)) if idx is None else list(idx[0, 0]) + [L - 1]
        o, ls, bound, lerr = tree_row(q64[0, 0], got[pos], SCALE)
        assert np.all(np.abs(out[0, 0].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB) + 1e-30)
        assert np.all(np.abs(lse[0, 0].double().cpu().numpy() - ls) <= lerr)


@pytest.mark.parametrize("H,ctx", [(16, 3000), (30, 3000), (60, 3000), (128, 3000)])
def test_a_wait_that_runs_out_ends_the_call(H, ctx):
    """The second tile's scores wait for a barrier that nothing signals, for 2 ms:
    every warp of every CTA gives up, the call returns with the error word set and
    the next call is right."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(14)
    paged = Paged(rng, [ctx, 700, 5], 64).fill(rng)
    q64, q = bf(rng.standard_normal((3, 1, H, DIM)))
    args = (q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), SCALE)
    X.tree_mla(*args, max_len=ctx)
    assert X.status() == (0, 0)
    X.debug_set(1, 2_000_000)
    try:
        X.tree_mla(*args, max_len=ctx)
        assert X.status() == (-7, X.DEV_ERR_TIMEOUT)
    finally:
        X.debug_set(0, 0)
    out, lse = X.tree_mla(*args, max_len=ctx)
    assert X.status() == (0, 0)
    check_tree(out, lse, q64, paged, [1, 1, 1], SCALE)
