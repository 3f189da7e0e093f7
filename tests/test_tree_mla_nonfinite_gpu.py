"""Drafts whose cache rows are not finite, in groups of rows that belong to several
tokens (idx_tree_mla): rows that do not see such a draft are as if it were not
there, rows that see it get what the definition gives, for every number of heads:

  score NaN or +inf: the weights are NaN, and so is everything;
  score −inf:        the weight is 0, and 0 · (what is not finite) = NaN stands in
                     the output features where the draft's row is not finite; the
                     others and lse are as without the draft."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, UB, Paged, bf, mask_dev, row_positions, tree_row

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
INF = float("inf")


def _call(X, paged, q, n, mask, dtype, indices=None, max_len=None):
    B, _, H = q.shape[:3]
    out = torch.full((B, n, H, LAT), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((B, n, H), 5.0, dtype=torch.float32, device="cuda")
    X.tree_mla(q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), SCALE,
               max_len=max_len or max(paged.lens), tree_mask=mask_dev(mask), out=out, lse=lse,
               indices=None if indices is None else dev(indices))
    assert X.status() == (0, 0)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _check(paged, q64, out, lse, n, mask, wild, bf16_out, indices=None):
    """wild: {(b, draft): features that are not finite}."""
    B, _, H = q64.shape[:3]
    for b in range(B):
        ctx = paged.lens[b] - n
        for i in range(n):
            seen = [j for j in range(n) if mask[b][i] >> j & 1 and (b, j) in wild]
            pos = row_positions(paged.lens, [n] * B, mask, indices, b, i)
            kv = paged.rows(b, paged.lens[b])
            with np.errstate(invalid="ignore"):
                s = np.array([[sum(q64[b, i, h, f] * kv[ctx + j][f] for f in wild[b, j]) for j in seen]
                              for h in range(H)]).reshape(H, len(seen))
            gone = np.any(np.isnan(s) | (s == INF), axis=1)      # heads whose weights are NaN
            o, ls, bound, lerr = tree_row(q64[b, i], kv[[t for t in pos if t - ctx not in seen]], SCALE)
            nan = np.zeros((H, LAT), bool)
            nan[gone] = True
            for j in seen:
                nan[:, [f for f in wild[b, j] if f < LAT]] = True
            got = out[b, i]
            assert np.array_equal(np.isnan(got), nan), (b, i, np.argwhere(np.isnan(got) != nan)[:4])
            bound = bound + (UB * np.abs(o) * (1 + UB) if bf16_out else 0) + 1e-30
            assert np.all(np.abs(got - o)[~nan] <= bound[~nan]), (b, i)
            assert np.array_equal(np.isnan(lse[b, i]), gone), (b, i)
            assert np.all(np.abs(lse[b, i] - ls)[~gone] <= lerr[~gone]), (b, i)


# heads, drafts: groups of 16, 32 and 64 rows, groups of 128 that cross tokens,
# and (last) groups of one token
SHAPES = [(4, 4), (10, 3), (16, 4), (16, 7), (20, 13), (128, 2)]
# context lengths: drafts across a tile's end (64 and 128 keys) in the first tiles and
# after the rings of tiles have gone round; few keys (items stay whole), many (they are cut)
CONTEXTS = [[126], [62, 190, 249], [900, 1150]]


def _case(seed, H, n, ctxs):
    rng = np.random.default_rng(seed)
    paged = Paged(rng, [c + n for c in ctxs], 48).fill(rng)
    q64, q = bf(rng.standard_normal((len(ctxs), n, H, DIM)))
    mask = [[(1 << i) | (1 if i % 2 else 0) for i in range(n)] for _ in ctxs]    # itself; odd rows the first, too
    return rng, paged, q64, q, mask


def _set(paged, n, b, j, features, value):
    t = paged.lens[b] - n + j
    paged.cache[paged.table[b, t // paged.page], t % paged.page, features] = value


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ctxs", CONTEXTS)
@pytest.mark.parametrize("H,n", SHAPES)
def test_one_feature_that_is_infinite(H, n, ctxs, dtype):
    """In the first half of the output features, the second, the rotary part: some
    heads score it −inf, others +inf."""
    from sparse_attention_token_idx_b200 import binding as X
    for f in (3, 300, 511, 520):
        _, paged, q64, _, mask = _case(H * 100 + f, H, n, ctxs)
        wild = {}
        for b in range(len(ctxs)):
            for j in {0, n - 1}:
                value = INF if (b + j) % 2 else -INF
                _set(paged, n, b, j, [f], value)
                wild[b, j] = [f]
                # most heads: −inf whichever row sees it; every third head +inf for one of the two
                q64[b, :, :, f] = np.where(np.arange(H) % 3 == 2, 1, -1) * np.sign(value) * (0.5 + np.abs(q64[b, :, :, f]))
        q64, q = bf(q64)
        out, lse = _call(X, paged, q, n, mask, dtype)
        _check(paged, q64, out, lse, n, mask, wild, dtype == torch.bfloat16)


@pytest.mark.parametrize("ctxs", CONTEXTS)
@pytest.mark.parametrize("H,n", SHAPES)
def test_nan_and_infinities_in_several_features(H, n, ctxs):
    from sparse_attention_token_idx_b200 import binding as X
    for fs, value in (([5], np.nan), ([10, 400], -INF), (list(range(DIM)), np.nan), ([575], np.nan)):
        _, paged, q64, _, mask = _case(H * 100 + len(fs), H, n, ctxs)
        wild = {}
        for b in range(len(ctxs)):
            _set(paged, n, b, n - 1, fs, value)
            wild[b, n - 1] = fs
        if value == -INF:
            q64[..., fs] = np.abs(q64[..., fs]) + 0.25
        q64, q = bf(q64)
        out, lse = _call(X, paged, q, n, mask, torch.float32)
        _check(paged, q64, out, lse, n, mask, wild, False)


def test_the_same_draft_through_different_numbers_of_heads():
    """A row's result does not depend on how many heads share the call."""
    from sparse_attention_token_idx_b200 import binding as X
    n, ctx = 3, 200
    _, paged, q64, _, mask = _case(5, 128, n, [ctx])
    _set(paged, n, 0, 1, [17, 333], -INF)
    q64[..., [17, 333]] = np.abs(q64[..., [17, 333]]) + 0.25
    q64, q = bf(q64)
    want, want_lse = _call(X, paged, q, n, mask, torch.float32)
    for H in (4, 10, 16, 30, 64):
        out, lse = _call(X, paged, q[:, :, :H].contiguous(), n, mask, torch.float32)
        assert np.array_equal(np.isnan(out), np.isnan(want[:, :, :H])) and np.isnan(out).any()
        assert np.array_equal(np.isnan(lse), np.isnan(want_lse[:, :, :H])) and not np.isnan(lse).any()


def test_a_selection_beside_such_a_draft():
    from sparse_attention_token_idx_b200 import binding as X
    for H, n in ((16, 4), (128, 2)):
        rng, paged, q64, _, mask = _case(H, H, n, [300])
        _set(paged, n, 0, 0, [40], INF)
        q64[..., 40] = -np.abs(q64[..., 40]) - 0.25
        q64, q = bf(q64)
        idx = np.stack([rng.choice(300, 90, replace=False) for _ in range(n)])[None].astype(np.int32)
        out, lse = _call(X, paged, q, n, mask, torch.float32, indices=idx)
        _check(paged, q64, out, lse, n, mask, {(0, 0): [40]}, False, indices=idx)


@pytest.mark.parametrize("H,n", SHAPES)
def test_rows_that_see_such_a_draft_alone(H, n):
    """No context: a row whose only key scores −inf has no weight to give."""
    from sparse_attention_token_idx_b200 import binding as X
    _, paged, q64, _, mask = _case(9, H, n, [0])
    mask = [[1 << i for i in range(n)]]
    _set(paged, n, 0, n - 1, [9], INF)
    q64[..., 9] = -np.abs(q64[..., 9]) - 0.25
    q64, q = bf(q64)
    out, lse = _call(X, paged, q, n, mask, torch.float32)
    assert np.isnan(out[0, n - 1, :, 9]).all() and not np.isfinite(lse[0, n - 1]).any()
    kv = paged.rows(0, n)
    for i in range(n - 1):
        o, ls, bound, lerr = tree_row(q64[0, i], kv[[i]], SCALE)
        assert np.all(np.abs(out[0, i] - o) <= bound + 1e-30) and np.all(np.abs(lse[0, i] - ls) <= lerr)


@pytest.mark.parametrize("H,n", [(10, 2), (16, 2), (10, 5), (16, 4), (8, 8), (20, 13)])
def test_fp32_output_of_drafted_rows_under_a_tree(H, n):
    """fp32 results of 17 to 64 rows (and more) that belong to several tokens, ragged,
    each token with a mask of its own."""
    from sparse_attention_token_idx_b200 import binding as X
    from tests.paged_helpers import check_tree, random_tree
    rng = np.random.default_rng(H * n)
    ctxs, cnts = [1500, 0, 133, 260], [n, n - 1, n, 1]
    paged = Paged(rng, [c + m for c, m in zip(ctxs, cnts)], 33).fill(rng)
    q64, q = bf(rng.standard_normal((4, n, H, DIM)))
    mask = [random_tree(rng, n) for _ in range(4)]
    mask[2][n - 1] = 0
    out = torch.full((4, n, H, LAT), 5.0, device="cuda")
    lse = torch.full((4, n, H), 5.0, device="cuda")
    X.tree_mla(q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), SCALE,
               max_len=max(paged.lens), counts=dev(np.array(cnts, np.int32)), tree_mask=mask_dev(mask), out=out, lse=lse)
    assert X.status() == (0, 0)
    check_tree(out, lse, q64, paged, cnts, SCALE, mask, untouched=5.0)
