"""Indexer.select: the selection of drafted rows over contexts of any length, none
among them, and what attention makes of it; byte scales; captured graphs beside
eager calls."""
import numpy as np
import pytest
import torch

from oracle import indexer as O
from tests.helpers import bf16_dev, check_topk_row, dev
from tests.paged_helpers import DIM, Paged, bf, check_tree

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16).numpy().view(np.uint16)


def _indexer(rng, ctxs, T_cap, fmt, k, scale_storage="f32"):
    """An Indexer that holds ctxs[b] keys of sequence b, and the oracle's cache of them."""
    from sparse_attention_token_idx_b200.pipeline import Indexer
    B = len(ctxs)
    ix = Indexer(B, T_cap, fmt, k, scale_storage=scale_storage)
    m = max(max(ctxs), 1)
    _, keys = bf(rng.standard_normal((B, m, 128)))
    ix.append(keys.cuda(), dev(np.zeros(B, np.int32)))
    kc, ks = np.zeros((B, T_cap, 128), np.uint8), np.zeros((B, T_cap), np.float32)
    O.quant_append(_bits(keys), [0] * B, kc, ks, fmt)
    return ix, kc, ks


def _queries(rng, B, n):
    _, q = bf(rng.standard_normal((B, n, 64, 128)))
    return q, rng.standard_normal((B, n, 64)).astype(np.float32)


def _check(got, q, w_raw, kc, ks, ctxs, fmt, k):
    codes, _, w = O.quant_queries(_bits(q), w_raw, fmt)
    for b, c in enumerate(ctxs):
        n = q.shape[1]
        if c == 0:
            assert np.all(got[b] == -1)
            continue
        S, E = O.index_scores_rows(codes[b], w[b], kc[b, :c], ks[b, :c], np.full(n, c))
        for i in range(n):
            check_topk_row(got[b, i], S[i], E[i], c, k)


@pytest.mark.parametrize("storage,fmt", [("f32", 0), ("f32", 1), ("e8m0", 1)])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 64])
def test_contexts_shorter_than_the_drafts(n, storage, fmt):
    """Every row of a sequence sees its whole context, however short: the decode
    route (one and two rows) and the workspace route."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(n)
    ctxs = [0, 1, max(n - 1, 0), n, 300, 2, 130]
    k = 16
    ix, kc, ks = _indexer(rng, ctxs, 512, fmt, k, storage)
    q, w_raw = _queries(rng, len(ctxs), n)
    lens = dev(np.array(ctxs, np.int32))
    for max_len in (max(ctxs), 512):
        idx = ix.select(q.cuda(), dev(w_raw), lens, max_len=max_len)
        assert X.status() == (0, 0)
        _check(idx.cpu().numpy(), q, w_raw, kc, ks, ctxs, fmt, k)


@pytest.mark.parametrize("n", [1, 8])
def test_no_sequence_has_more_context_than_drafts(n):
    """The first steps of a batch: the host bound is below the number of drafts, or 0."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(40 + n)
    for ctxs in ([0, 0], [1, 0], [3, 2]):
        ix, kc, ks = _indexer(rng, ctxs, 64, 0, 8)
        q, w_raw = _queries(rng, 2, n)
        idx = ix.select(q.cuda(), dev(w_raw), dev(np.array(ctxs, np.int32)), max_len=max(ctxs))
        assert X.status() == (0, 0)
        _check(idx.cpu().numpy(), q, w_raw, kc, ks, ctxs, 0, 8)


def test_lengths_out_of_range_are_reported():
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(50)
    ix, kc, ks = _indexer(rng, [40, 40, 40], 64, 0, 8)
    for n in (1, 8):
        q, w_raw = _queries(rng, 3, n)
        for bad in (-1, 41, -2147483648):
            idx = ix.select(q.cuda(), dev(w_raw), dev(np.array([bad, 40, 5], np.int32)), max_len=40)
            assert X.status() == (-7, X.DEV_ERR_LENGTH)
            got = idx.cpu().numpy()
            assert np.all(got[0] == -1)
            _check(got[1:], q[1:], w_raw[1:], kc[1:], ks[1:], [40, 5], 0, 8)


def test_causal_calls_still_need_their_rows():
    """Rows that are cached themselves: fewer keys than rows is an error, as it was."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(51)
    ix, _, _ = _indexer(rng, [5, 40], 64, 0, 8)
    q, w_raw = _queries(rng, 2, 8)
    codes, w = X.quant_queries(q.cuda(), dev(w_raw), 0)
    lens = dev(np.array([5, 40], np.int32))
    idx = X.score_topk(codes, w, ix.k_cache, ix.k_scale_cache, lens, True, 8, 40)
    assert X.status() == (-7, X.DEV_ERR_LENGTH) and bool((idx[0] == -1).all())
    with pytest.raises(X.IdxError):
        X.score_topk(codes, w, ix.k_cache, ix.k_scale_cache, lens, True, 8, 7)   # max_len < n


def test_scores_of_short_contexts():
    """The score calls themselves, rows not cached: valid up to the context, −inf behind it."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(52)
    ctxs = [0, 3, 70]
    ix, kc, ks = _indexer(rng, ctxs, 128, 0, 8)
    q, w_raw = _queries(rng, 3, 8)
    codes, w = X.quant_queries(q.cuda(), dev(w_raw), 0)
    s = X.score(codes, w, ix.k_cache, ix.k_scale_cache, dev(np.array(ctxs, np.int32)), False, 128).cpu().numpy()
    assert X.status() == (0, 0)
    qc, _, wf = O.quant_queries(_bits(q), w_raw, 0)
    for b, c in enumerate(ctxs):
        assert np.all(np.isneginf(s[b, :, c:]))
        if c:
            S, E = O.index_scores_rows(qc[b], wf[b], kc[b, :c], ks[b, :c], np.full(8, c))
            assert np.all(np.abs(s[b, :, :c] - S) <= 1e-5 * E)


def test_selection_then_attention_at_the_start_of_sequences():
    """Drafts behind contexts of 0, 1, n − 1 and more positions attend to all of a
    short context, and to the selection of a long one."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(53)
    n, H, k = 8, 16, 32
    ctxs, cnts = [0, 1, 7, 200], [8, 5, 8, 2]
    ix, _, _ = _indexer(rng, ctxs, 256, 0, k)
    iq, w_raw = _queries(rng, 4, n)
    idx = ix.select(iq.cuda(), dev(w_raw), dev(np.array(ctxs, np.int32)), max_len=200)
    got = idx.cpu().numpy()
    for b in range(3):
        for i in range(n):
            assert sorted(t for t in got[b, i] if t >= 0) == list(range(ctxs[b]))
    paged = Paged(rng, [c + m for c, m in zip(ctxs, cnts)], 16).fill(rng)
    q64, q = bf(rng.standard_normal((4, n, H, DIM)))
    out, lse = X.tree_mla(q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), 0.07,
                          max_len=max(paged.lens), counts=dev(np.array(cnts, np.int32)), indices=idx)
    assert X.status() == (0, 0)
    check_tree(out, lse, q64, paged, cnts, 0.07, None, got)
