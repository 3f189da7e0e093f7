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


def test_select_refuses_shapes_that_are_not_its_caches():
    import torch
    from sparse_attention_token_idx_b200.pipeline import Indexer
    ix = Indexer(2, 64, 0, 16, device="cpu")
    z, bf, i32 = torch.zeros, torch.bfloat16, torch.int32

    def select(q=(2, 3, 64, 128), w=(2, 3, 64), n=(2,), out=None):
        return ix.select(z(q, dtype=bf), z(w), z(n, dtype=i32), max_len=64, out=out)

    for kw in (dict(q=(3, 3, 64, 128), w=(3, 3, 64), n=(3,)), dict(q=(2, 3, 64, 128), w=(1, 3, 64)),
               dict(q=(2, 3, 32, 128)), dict(q=(2, 3, 64, 64)), dict(w=(2, 64)), dict(w=(2, 2, 64)), dict(n=(3,)),
               dict(n=(2, 1)), dict(out=z((2, 3, 8), dtype=i32)), dict(out=z((2, 2, 16), dtype=i32))):
        with pytest.raises(ValueError):
            select(**kw)


def test_select_runs_on_its_caches_device_and_the_calls_stream(monkeypatch):
    """Whichever device is the current one: the library's calls are made with the
    cache's as the current one, and on the stream that was given."""
    import contextlib
    import torch
    from sparse_attention_token_idx_b200 import pipeline
    from sparse_attention_token_idx_b200.pipeline import Indexer
    X, at, made = pipeline.X, [(0, None)], []

    @contextlib.contextmanager
    def entered(device, stream):
        at.append((device, stream))
        yield
        at.pop()

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(X, "_on", entered)
    monkeypatch.setattr(X, "_current_device", lambda: at[-1][0])
    monkeypatch.setattr(X, "_current_stream", lambda device: 7)
    monkeypatch.setattr(X, "workspace_size", lambda *a: 0)
    monkeypatch.setattr(X, "quant_queries", lambda *a, stream=None: made.append((at[-1], stream)))
    monkeypatch.setattr(X, "score_topk_ex", lambda *a, out, ws, stream=None: made.append((at[-1], stream)))
    ix = Indexer(2, 64, 0, 16, device="cpu")
    ix._index = 3
    z = torch.zeros
    a = (z((2, 3, 64, 128), dtype=torch.bfloat16), z((2, 3, 64)), z(2, dtype=torch.int32))
    for stream in (None, "a stream"):
        made.clear()
        ix.select(*a, max_len=64, stream=stream)
        assert made == [((3, stream), None)] * 2
    at[0] = (3, None)                                            # nothing to switch
    made.clear()
    ix.select(*a, max_len=64)
    assert made == [((3, None), None)] * 2 and len(at) == 1
