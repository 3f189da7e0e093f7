"""The paged operators together, as a speculative decode step uses them: prompts
appended in chunks, a tree of drafts appended with its depths as positions, its
rows attended to over the whole context and over an indexer's selection of it."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, UB, bf, mask_dev, random_tree, tree_row

pytestmark = pytest.mark.gpu


def _tables(pos):
    freq = 10000.0 ** (-np.arange(32) / 32)
    ang = np.asarray(pos, np.float64)[..., None] * freq
    return dev(np.cos(ang).astype(np.float32)), dev(np.sin(ang).astype(np.float32))


def _rows_of(lc, b, L):
    t = torch.arange(L)
    return lc.cache[lc._table[b].long()[t // lc.page_size].cuda(), (t % lc.page_size).cuda()].double().cpu().numpy()


def test_prompt_drafts_and_attention():
    from sparse_attention_token_idx_b200 import binding as X
    from sparse_attention_token_idx_b200.pipeline import Indexer, LatentCache
    rng = np.random.default_rng(21)
    B, H, page, n, k, scale = 3, 16, 32, 6, 64, 192 ** -0.5
    ctxs, cnts = [300, 77, 130], [6, 3, 5]
    lc = LatentCache(B, 40, page, 512)
    gain = dev((1 + 0.1 * rng.standard_normal(LAT)).astype(np.float32))
    for b in range(B):
        lc.reserve(b, ctxs[b] + cnts[b])
    # prompts, 128 tokens a chunk, ragged
    for start in range(0, max(ctxs), 128):
        m = [max(0, min(128, c - start)) for c in ctxs]
        _, kv = bf(rng.standard_normal((B, 128, DIM)))
        cos, sin = _tables(np.tile(start + np.arange(128), (B, 1)))
        lc.append(kv.cuda(), gain, 1e-6, cos, sin, dev(np.full(B, start, np.int32)), counts=dev(np.array(m, np.int32)))
    before = [_rows_of(lc, b, ctxs[b]) for b in range(B)]
    # drafts: slots behind the context, positions by depth
    trees = [random_tree(rng, n) for _ in range(B)]
    depth = [[bin(r).count("1") - 1 for r in row] for row in trees]
    _, kv = bf(rng.standard_normal((B, n, DIM)))
    _, q = bf(rng.standard_normal((B, n, H, DIM)))
    q = q.cuda()
    q_pe = q[..., LAT:].clone()
    cos, sin = _tables(np.array(ctxs)[:, None] + np.array(depth))
    lc.append(kv.cuda(), gain, 1e-6, cos, sin, dev(np.array(ctxs, np.int32)), counts=dev(np.array(cnts, np.int32)),
              q_pe=q_pe, q_out=q)
    lens = dev(np.array([a + c for a, c in zip(ctxs, cnts)], np.int32))
    rows = [_rows_of(lc, b, ctxs[b] + cnts[b]) for b in range(B)]
    for b in range(B):
        assert np.array_equal(rows[b][:ctxs[b]], before[b])      # the context is as it was
    qn = q.double().cpu().numpy()

    def check(out, lse, idx=None):
        assert X.status() == (0, 0)
        for b in range(B):
            for i in range(cnts[b]):
                pos = list(range(ctxs[b])) if idx is None else [int(t) for t in idx[b, i] if t >= 0]
                pos += [ctxs[b] + j for j in range(cnts[b]) if trees[b][i] >> j & 1]
                o, ls, bound, lerr = tree_row(qn[b, i], rows[b][pos], scale)
                assert np.all(np.abs(out[b, i].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB) + 1e-30)
                assert np.all(np.abs(lse[b, i].double().cpu().numpy() - ls) <= lerr)

    kw = dict(counts=dev(np.array(cnts, np.int32)), tree_mask=mask_dev(trees))
    check(*lc.attend(q, lens, scale, **kw))
    # the indexer's keys of the context, and its selection for every drafted row
    ix = Indexer(B, 512, 0, k)
    for b in range(B):
        _, ik = bf(rng.standard_normal((1, ctxs[b], 128)))
        X.quant_append(ik.cuda(), dev(np.zeros(1, np.int32)), ix.k_cache[b:b + 1], ix.k_scale_cache[b:b + 1], 0)
    _, iq = bf(rng.standard_normal((B, n, 64, 128)))
    w = dev(rng.standard_normal((B, n, 64)).astype(np.float32))
    idx = ix.select(iq.cuda(), w, dev(np.array(ctxs, np.int32)), max_len=max(ctxs))
    got = idx.cpu().numpy()
    for b in range(B):
        for i in range(n):
            sel = got[b, i][got[b, i] >= 0]
            assert len(sel) == min(k, ctxs[b]) == len(set(sel.tolist())) and sel.max() < ctxs[b]
    check(*lc.attend(q, lens, scale, indices=idx, **kw), idx=got)


def test_a_captured_step_replays_on_new_inputs():
    """Append and attend captured in one graph, replayed after the inputs changed
    in place: the same bits as the calls made eagerly."""
    from sparse_attention_token_idx_b200.pipeline import LatentCache
    rng = np.random.default_rng(22)
    B, H, L = 4, 128, 700
    caches = [LatentCache(B, 60, 64, 1024) for _ in range(2)]
    gain = dev(np.ones(LAT, np.float32))
    for lc in caches:
        for b in range(B):
            lc.reserve(b, L + 3)
    _, kv0 = bf(rng.standard_normal((B, L, DIM)))
    cos0, sin0 = _tables(np.tile(np.arange(L), (B, 1)))
    for lc in caches:
        lc.append(kv0.cuda(), gain, 1e-6, cos0, sin0, dev(np.zeros(B, np.int32)))
    kv = torch.zeros((B, 1, DIM), dtype=torch.bfloat16, device="cuda")
    q_pe = torch.zeros((B, 1, H, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((B, 1, H, DIM), dtype=torch.bfloat16, device="cuda")
    pos, lens = dev(np.full(B, L, np.int32)), dev(np.full(B, L + 1, np.int32))
    cos, sin = (t.clone() for t in _tables(np.full((B, 1), L)))
    out = torch.zeros((B, 1, H, LAT), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((B, 1, H), device="cuda")

    def step(lc, o, s):
        lc.append(kv, gain, 1e-6, cos, sin, pos, q_pe=q_pe, q_out=q)
        lc.attend(q, lens, 0.07, max_len=1024, out=o, lse=s)

    step(caches[1], torch.zeros_like(out), torch.zeros_like(lse))   # warm-up: kernels loaded, workspace made
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(caches[1], out, lse)
    for i in range(3):
        kv.copy_(bf(rng.standard_normal((B, 1, DIM)))[1])
        q_pe.copy_(bf(rng.standard_normal((B, 1, H, 64)))[1])
        q[..., :LAT].copy_(bf(rng.standard_normal((B, 1, H, LAT)))[1])
        for t, v in ((pos, L + i), (lens, L + i + 1)):
            t.fill_(v)
        c, s = _tables(np.full((B, 1), L + i))
        cos.copy_(c)
        sin.copy_(s)
        want, want_lse = torch.zeros_like(out), torch.zeros_like(lse)
        step(caches[0], want, want_lse)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
