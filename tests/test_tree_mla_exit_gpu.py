"""The way out of idx_tree_mla when a warp gives up where its CTA's work has ended:
the warps that share its rows have met for the last time by then, and come to one
more meeting before they go.  Every wait here ends after 2 ms."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, Paged, bf, check_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [4, 16, 30, 60, 128])
@pytest.mark.parametrize("lens,max_len", [
    ([3000, 700, 5], 3000),       # items cut over many CTAs
    ([40, 3], 5000),              # most CTAs have an empty share
    ([200, 130, 64, 1], 256),     # items stay whole
])
def test_a_warp_that_gives_up_at_the_end_of_the_list(H, lens, max_len):
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(H)
    B = len(lens)
    paged = Paged(rng, lens, 64, width=-(-max_len // 64)).fill(rng)
    q64, q = bf(rng.standard_normal((B, 1, H, DIM)))
    args = (q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(lens, np.int32)), 0.07)
    want, want_lse = X.tree_mla(*args, max_len=max_len)
    assert X.status() == (0, 0)
    check_tree(want, want_lse, q64, paged, [1] * B, 0.07)
    for flags in (4, 5):                                         # alone; beside scores that wait for nothing
        X.debug_set(flags, 2_000_000)
        try:
            out, lse = X.tree_mla(*args, max_len=max_len)
            assert X.status() == (-7, X.DEV_ERR_TIMEOUT)
        finally:
            X.debug_set(0, 0)
        if flags == 4:                                           # the results were written before
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
        out, lse = X.tree_mla(*args, max_len=max_len)
        assert X.status() == (0, 0) and torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("H", [16, 30, 60, 128])
def test_what_is_in_flight_is_waited_for_whatever_the_budget(H):
    """A budget of 100 us: CTAs give up in mid-work one after another; copies and
    products in flight end before their memory goes back, and the next call is right."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(H + 1)
    paged = Paged(rng, [3000, 700, 5], 64).fill(rng)
    q64, q = bf(rng.standard_normal((3, 1, H, DIM)))
    args = (q.cuda(), paged.cache_dev(), paged.table_dev(), dev(np.array(paged.lens, np.int32)), 0.07)
    want, want_lse = X.tree_mla(*args, max_len=3000)
    assert X.status() == (0, 0)
    for _ in range(20):
        X.debug_set(1, 100_000)
        try:
            X.tree_mla(*args, max_len=3000)
            assert X.status() == (-7, X.DEV_ERR_TIMEOUT)
        finally:
            X.debug_set(0, 0)
        out, lse = X.tree_mla(*args, max_len=3000)
        assert X.status() == (0, 0) and torch.equal(out, want) and torch.equal(lse, want_lse)
