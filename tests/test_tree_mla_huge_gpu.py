"""Scores far beyond what a softmax can tell apart (idx_tree_mla): each is one exact
product, the largest ones of a row are equal and all others are lower by more than
the exponential can hold, so the row's output is the mean of the latent features of
the positions with the largest score, and lse that score (plus ln of their number).

Bounds: equal weights are equal as computed, so the output is a mean of at most 8
bf16 numbers: the weight's rounding (2^-8, twice: above the division only), fp32
sums (8 + 600 roundings of 2^-24) and the output's rounding (2^-8).  lse: the scale
times log2 e, the product with the score, and the product with ln 2, each rounded
once, and the constants: 8 · 2^-24 of the score."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, U, UB, Paged, bf

pytestmark = pytest.mark.gpu


def _rows(rng, L, factor, rising):
    """Integer scores (their multiple of `factor`): below 0 … −199, the largest, −1,
    at a few places; rising: the largest so far grows along the sequence."""
    a = -2.0 - rng.integers(0, 150, L)
    if rising:
        a = -200.0 + np.floor(150 * np.arange(L) / max(L, 2))
    top = rng.choice(L, min(L, 3), replace=False)
    a[top] = -1.0
    return a * factor, np.sort(top)


@pytest.mark.parametrize("H", [3, 30, 60, 128])
@pytest.mark.parametrize("L,max_len", [(100, 100), (250, 250), (700, 700), (3000, 3000)])
@pytest.mark.parametrize("factor,scale", [(2.0 ** 20, 1.0), (2.0 ** 31, 0.7), (2.0 ** 60, -1.3), (2.0 ** 110, 0.07),
                                          (2.0 ** 126.5, 0.8)])
def test_rows_are_the_mean_of_their_best_positions(H, L, max_len, factor, scale):
    from sparse_attention_token_idx_b200 import binding as X
    for rising in (False, True):
        rng = np.random.default_rng(L + H)
        paged = Paged(rng, [L, L // 2 + 1], 64).fill(rng)
        tops, most = [], []
        sq = 2.0 ** int(np.log2(factor) / 2)                     # the query's share of the factor
        for b, n in enumerate(paged.lens):
            a, top = _rows(rng, n, factor / sq if factor < 2.0 ** 126 else 1.0, rising)
            if factor > 2.0 ** 126:                              # scores that fill the range: the best is −2.2e38
                a = np.where(a == -1.0, -2.2e38, -3.2e38) / sq
            for t in range(n):
                row = paged.cache[paged.table[b, t // 64], t % 64]
                row[LAT:] = 0
                row[LAT + 7] = a[t]
            paged.cache[:] = bf(paged.cache)[0]
            kv = paged.rows(b, n)[:, LAT + 7]
            best = np.flatnonzero(kv == kv.max())
            tops.append(best)
            most.append(kv.max())
        q = np.zeros((2, 1, H, DIM))
        q[..., LAT + 7] = sq * np.sign(scale)
        _, qt = bf(q)
        out, lse = X.tree_mla(qt.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), scale,
                              max_len=max_len, out=torch.empty((2, 1, H, LAT), device="cuda"))
        assert X.status() == (0, 0)
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(2):
            v = paged.rows(b, paged.lens[b])[tops[b]][:, :LAT]
            want = v.mean(axis=0)
            assert np.all(np.abs(got[b] - want) <= np.abs(v).mean(axis=0) * (2 * UB + 700 * U)), (b, rising)
            s = most[b] * sq * abs(scale) + np.log(len(tops[b]))
            assert np.all(np.abs(gl[b] - s) <= 8 * U * abs(s)), (b, rising)


@pytest.mark.parametrize("H", [3, 30, 60, 128])
def test_a_lowest_score_after_keys_that_are_not_there(H):
    """A selection whose first tiles are empty, then positions whose score is near the
    lowest number: the row sees them."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(H)
    for value in (-2.2e38, -2.07e38, -1e38, -3.0):
        paged = Paged(rng, [301], 64).fill(rng)
        kv = paged.cache
        kv[..., LAT:] = np.where(np.isnan(kv[..., LAT:]), np.nan, 0)
        kv[..., LAT + 1] = np.where(np.isnan(kv[..., LAT + 1]), np.nan, bf(np.full(1, value))[0][0])
        q = np.zeros((1, 1, H, DIM))
        q[..., LAT + 1] = 1
        _, qt = bf(q)
        for lead in (128, 150, 300):
            idx = np.full((1, 1, lead + 4), -1, np.int32)
            idx[0, 0, lead:] = [5, 250, 130, 77]
            out, lse = X.tree_mla(qt.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array([301], np.int32)), 1.0,
                                  max_len=301, indices=dev(idx), tree_mask=torch.zeros((1, 1), dtype=torch.int64, device="cuda"),
                                  out=torch.empty((1, 1, H, LAT), device="cuda"))
            assert X.status() == (0, 0)
            v = paged.rows(0, 301)[[5, 250, 130, 77], :LAT]
            got = out[0, 0].double().cpu().numpy()
            assert np.all(np.abs(got - v.mean(axis=0)) <= np.abs(v).mean(axis=0) * (2 * UB + 700 * U)), (value, lead)
            s = bf(np.full(1, value))[0][0] + np.log(4)
            assert np.all(np.abs(lse[0, 0].double().cpu().numpy() - s) <= 8 * U * abs(s)), (value, lead)


@pytest.mark.parametrize("H", [3, 30, 60, 128])
def test_scores_beyond_the_range_count_as_infinite(H):
    """−2.9e38 weighs nothing, beside other scores and alone; +2.9e38 is not a number's."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(H)
    for L in (90, 900):
        paged = Paged(rng, [L], 64).fill(rng)
        kv = paged.cache
        kv[..., LAT:] = np.where(np.isnan(kv[..., LAT:]), np.nan, 0)
        kv[..., LAT + 1] = np.where(np.isnan(kv[..., LAT + 1]), np.nan, bf(np.full(1, -2.2e38))[0][0])
        q = np.zeros((1, 1, H, DIM))
        q[..., LAT + 1] = 1
        _, qt = bf(q)

        def go(scale):
            out, lse = X.tree_mla(qt.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array([L], np.int32)), scale,
                                  max_len=L, out=torch.empty((1, 1, H, LAT), device="cuda"))
            assert X.status() == (0, 0)
            return out[0, 0].double().cpu().numpy(), lse[0, 0].double().cpu().numpy()

        out, lse = go(1.3)
        assert np.all(out == 0) and np.all(lse == -np.inf)
        out, lse = go(-1.3)
        assert np.all(np.isnan(out)) and not np.isfinite(lse).any()
        ordinary = [3, L // 2, L - 1]
        for t in ordinary:
            kv[paged.table[0, t // 64], t % 64, LAT + 1] = 4.0
        out, lse = go(1.3)
        v = paged.rows(0, L)[ordinary][:, :LAT]
        assert np.all(np.abs(out - v.mean(axis=0)) <= np.abs(v).mean(axis=0) * (2 * UB + 700 * U))
        assert np.all(np.abs(lse - (5.2 + np.log(3))) <= 1e-5)
