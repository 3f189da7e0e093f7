"""Captured indexer calls beside eager ones of other shapes: replays give what the
eager call gives and write into nobody else's memory."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import bf

pytestmark = pytest.mark.gpu

B, T_CAP, K, CTX = 3, 2048, 64, 1500


def _indexer(rng):
    from sparse_attention_token_idx_b200.pipeline import Indexer
    ix = Indexer(B, T_CAP, 0, K)
    _, keys = bf(rng.standard_normal((B, CTX, 128)))
    ix.append(keys.cuda(), dev(np.zeros(B, np.int32)))
    return ix


def _queries(rng, n):
    _, q = bf(rng.standard_normal((B, n, 64, 128)))
    return q.cuda(), dev(rng.standard_normal((B, n, 64)).astype(np.float32))


def _fills():
    """Tensors of many sizes, each full of one byte: what the allocator has to give away."""
    return [torch.full((s,), 0xA5, dtype=torch.uint8, device="cuda")
            for s in (512, 4096, 24576, 65536, 200000, 196608, 1 << 20, 1572864, 3 << 20, 1 << 22, 1 << 24) for _ in range(6)]


def _sets(t):
    return torch.sort(t, -1).values


def test_captured_step_and_selections_beside_eager_calls():
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(61)
    ix = _indexer(rng)
    lens = dev(np.full(B, CTX, np.int32))
    pos, lens1 = dev(np.full(B, CTX, np.int32)), dev(np.full(B, CTX + 1, np.int32))     # (a graph's inputs stay alive)
    q1, w1 = _queries(rng, 1)
    _, k1 = bf(rng.standard_normal((B, 1, 128)))
    k1 = k1.cuda()
    sel_in = {n: _queries(rng, n) for n in (1, 8, 40)}
    g_step, out_step = ix.capture(k1, q1, w1, pos, lens1, causal=False, max_len=T_CAP)
    graphs = {}
    for n, (q, w) in sel_in.items():
        ix.select(q, w, lens, max_len=T_CAP)                     # warm-up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ix.select(q, w, lens, max_len=T_CAP)
        graphs[n] = (g, out)
    # eager calls of other shapes, whose scratch replaces what was kept, then new tensors
    for n in (2, 16, 70):
        q, w = _queries(rng, n)
        _, k = bf(rng.standard_normal((B, n, 128)))
        ix.step(k.cuda(), q, w, pos, lens + n, causal=True, max_len=T_CAP)
        ix.select(q, w, lens, max_len=CTX + n)
    torch.cuda.synchronize()
    fills = _fills()
    torch.cuda.synchronize()
    for _ in range(2):
        g_step.replay()
        for g, _ in graphs.values():
            g.replay()
    torch.cuda.synchronize()
    assert X.status() == (0, 0)
    assert all(bool((f == 0xA5).all()) for f in fills)
    for n, (q, w) in sel_in.items():
        want = ix.select(q, w, lens, max_len=T_CAP)
        assert torch.equal(_sets(graphs[n][1]), _sets(want))
    got = out_step.clone()
    want = ix.step(k1, q1, w1, pos, lens1, causal=False, max_len=T_CAP)
    assert torch.equal(_sets(got), _sets(want))


def test_graphs_of_one_shape_replayed_at_once():
    """Two captures of one indexer on their own streams: no scratch in common."""
    rng = np.random.default_rng(62)
    ix = _indexer(rng)
    lens = dev(np.full(B, CTX, np.int32))
    ins = [_queries(rng, 40) for _ in range(2)]
    want = [_sets(ix.select(q, w, lens, max_len=T_CAP)) for q, w in ins]
    torch.cuda.synchronize()
    graphs = []
    for q, w in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ix.select(q, w, lens, max_len=T_CAP)
        graphs.append((g, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (g, out, s), ref in zip(graphs, want):
        assert torch.equal(_sets(out), ref)


def test_results_stay_the_callers():
    """What step and select returned is not written by the other."""
    rng = np.random.default_rng(63)
    ix = _indexer(rng)
    lens = dev(np.full(B, CTX, np.int32))
    q, w = _queries(rng, 8)
    q2, w2 = _queries(rng, 8)
    _, k = bf(rng.standard_normal((B, 8, 128)))
    first = ix.select(q, w, lens, max_len=T_CAP)
    kept = first.clone()
    stepped = ix.step(k.cuda(), q2, w2, lens, lens + 8, causal=True, max_len=T_CAP)
    kept_step = stepped.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ix.select(q2, w2, lens, max_len=T_CAP, stream=s)
    s.synchronize()
    assert torch.equal(first, kept) and torch.equal(stepped, kept_step)
