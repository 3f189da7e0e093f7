"""Who holds the Indexer's scratch (host logic, on CPU tensors with the library's
calls replaced): a selection takes none of a step's, and what a capture has seen
belongs to no later call."""
import pytest
import torch

from sparse_attention_token_idx_b200 import pipeline
from sparse_attention_token_idx_b200.pipeline import Indexer


class Calls:
    """Stand-ins for the library's calls; keeps the tensors that each was given."""

    def __init__(self, monkeypatch):
        self.capturing, self.seen = False, []
        X = pipeline.X
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(X, "workspace_size", lambda B, n, max_len, k: B * n * max_len * 4 if n > 2 else 0)
        monkeypatch.setattr(X, "project_workspace_size", lambda T, hidden, q_lora: 16 * T)
        monkeypatch.setattr(X, "quant_queries", lambda q, w, fmt, q8, wf, stream=None: self.keep(q8, wf))
        monkeypatch.setattr(X, "quant_queries_append",
                            lambda q, w, k, p, kc, ks, fmt, q8, wf, stream=None: self.keep(q8, wf))
        monkeypatch.setattr(X, "front_quant_append", lambda *a, stream=None: self.keep(a[-2], a[-1]))
        monkeypatch.setattr(X, "project", lambda *a, q_out, k_out, w_out, ws, stream=None:
                            self.keep(q_out, k_out, w_out, ws))

        def topk(q8, w, kc, ks, lengths, causal, k, max_len, out, ws, stream=None):
            self.keep(q8, w, out, ws)
            return out

        monkeypatch.setattr(X, "score_topk_ex", topk)

    def keep(self, *tensors):
        self.seen += [t for t in tensors if t is not None]

    def storages(self, call):
        """Storages that `call` hands to the library (all kept alive here, so that no two agree by reuse)."""
        at = len(self.seen)
        result = call()
        return {t.untyped_storage().data_ptr() for t in self.seen[at:]}, result


def _args(n):
    z = torch.zeros
    return dict(q=z((2, n, 64, 128), dtype=torch.bfloat16), w_raw=z((2, n, 64)), lengths=z(2, dtype=torch.int32))


def _step(ix, n):
    a = _args(n)
    return ix.step(torch.zeros((2, n, 128), dtype=torch.bfloat16), a["q"], a["w_raw"], a["lengths"], a["lengths"],
                   causal=False, max_len=64)


def _select(ix, n):
    return ix.select(**_args(n), max_len=64)


def _hidden(ix, n):
    z, bf = torch.zeros, torch.bfloat16
    return ix.step_hidden(z((2, n, 32), dtype=bf), z((2, n, 16), dtype=bf), z((8192, 16), dtype=bf), z((128, 32), dtype=bf),
                          z((64, 32)), z((2, n, 32)), z((2, n, 32)), z(128), z(128), z(2, dtype=torch.int32),
                          z(2, dtype=torch.int32), causal=False, max_len=64)


@pytest.mark.parametrize("n", [1, 8])
def test_a_selection_and_a_step_of_one_shape_share_nothing(monkeypatch, n):
    calls, ix = Calls(monkeypatch), Indexer(2, 64, 0, 16, device="cpu")
    step, idx = calls.storages(lambda: _step(ix, n))
    select, sel = calls.storages(lambda: _select(ix, n))
    assert idx is not sel and not step & select
    again, sel2 = calls.storages(lambda: _select(ix, n))
    assert sel2 is not sel                                       # a result is the caller's to keep
    assert again & select == select - {sel.untyped_storage().data_ptr()}   # the scratch stays where it was
    assert calls.storages(lambda: _step(ix, n))[0] == step       # a step's scratch stays where it was


@pytest.mark.parametrize("n", [1, 8])
@pytest.mark.parametrize("captured", [_step, _select, _hidden])
def test_what_a_capture_uses_is_its_own(monkeypatch, captured, n):
    calls, ix = Calls(monkeypatch), Indexer(2, 64, 0, 16, device="cpu")
    eager, _ = calls.storages(lambda: captured(ix, n))           # the warm-up of a capture
    calls.capturing = True
    graph, _ = calls.storages(lambda: captured(ix, n))
    graph2, _ = calls.storages(lambda: captured(ix, n))
    calls.capturing = False
    after = set()
    for call, m in ((_select, 8), (_step, 8), (_step, 1), (_hidden, 8), (_hidden, 1), (_select, n), (captured, n)):
        after |= calls.storages(lambda: call(ix, m))[0]
    assert not graph & (eager | after) and not graph2 & (eager | after | graph)


def test_projections_are_those_of_the_last_call(monkeypatch):
    calls, ix = Calls(monkeypatch), Indexer(2, 64, 0, 16, device="cpu")
    for n in (1, 8, 1):
        _hidden(ix, n)
        q, k, w = ix.projections()
        assert q.shape == (2, n, 64, 128) and k.shape == (2, n, 128) and w.shape == (2, n, 64)
    calls.capturing = True
    graph, _ = calls.storages(lambda: _hidden(ix, 1))
    assert {t.untyped_storage().data_ptr() for t in ix.projections()} <= graph


def test_scratch_belongs_to_one_stream(monkeypatch):
    """A call on another stream does not take what a call on the first may still use."""
    import contextlib
    from types import SimpleNamespace
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    calls, ix = Calls(monkeypatch), Indexer(2, 64, 0, 16, device="cpu")
    one, two = SimpleNamespace(cuda_stream=11), SimpleNamespace(cuda_stream=12)
    a = _args(8)
    used = [calls.storages(lambda: ix.select(**a, max_len=64, stream=s, out=torch.zeros((2, 8, 16), dtype=torch.int32)))[0]
            for s in (one, one, two, two)]
    out = [t.untyped_storage().data_ptr() for t in calls.seen if t.shape == (2, 8, 16)]
    used = [u - set(out) for u in used]
    assert used[0] == used[1] and used[2] == used[3] and not used[0] & used[2]
