"""Host checks of the score and top-k calls on the bound of the lengths (dummy
addresses that are never dereferenced; every call here is refused)."""
import pytest

P16 = 1 << 20
SHAPE = -2


@pytest.mark.parametrize("n,max_len,causal", [(8, 7, 1), (1, 0, 1), (1, 0, 0), (8, 0, 0), (8, -1, 0), (8, 65, 0), (8, 65, 1),
                                              (8, 16, 2)])
def test_bounds_that_are_refused(n, max_len, causal):
    from sparse_attention_token_idx_b200 import binding
    lib = binding.load()
    assert lib.idx_score_topk(P16, P16, P16, P16, P16, 2, n, 64, max_len, causal, 8, P16, None, 0, None) == SHAPE
    assert lib.idx_score(P16, P16, P16, P16, P16, 2, n, 64, max_len, causal, P16, 64, None) == SHAPE
    assert lib.idx_topk(P16, P16, 2, n, 64, max_len, causal, 8, P16, None, 0, None) == SHAPE
