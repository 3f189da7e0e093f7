"""Page bookkeeping of LatentCache (host logic, on CPU tensors)."""
import pytest
import torch

from sparse_attention_token_idx_b200 import binding as X
from sparse_attention_token_idx_b200.pipeline import LatentCache


def test_pages_are_reserved_released_and_shared():
    c = LatentCache(3, 6, 16, 64, device="cpu")
    assert c.max_pages == 4 and (c.table() == -1).all()
    c.reserve(0, 33)                                             # three pages
    c.reserve(0, 20)                                             # nothing more
    t = c.table()
    held = t[0, :3].tolist()
    assert len(set(held)) == 3 and t[0, 3] == -1 and (t[1:] == -1).all()
    assert c.share(1, 0, 40) == 32                               # whole pages only
    assert c.table()[1, :2].tolist() == held[:2]
    c.reserve(1, 48)
    assert c.table()[1, 2].item() not in held
    c.release(0)                                                 # its third page is free again, the shared ones are not
    c.reserve(2, 48)
    assert not set(c.table()[2, :3].tolist()) & set(c.table()[1, :3].tolist())
    with pytest.raises(X.IdxError):
        c.reserve(0, 1)                                          # none left
    c.release(1)
    c.release(2)
    assert sorted(c._free) == list(range(6)) and c._users == [0] * 6


def test_sequences_and_lengths_out_of_range_are_refused():
    c = LatentCache(2, 6, 16, 64, device="cpu")
    c.reserve(1, 48)
    for call in (lambda: c.share(0, 1, -1), lambda: c.share(0, 2, 16), lambda: c.share(-1, 0, 16),
                 lambda: c.reserve(-1, 16), lambda: c.reserve(2, 16), lambda: c.reserve(0, -1),
                 lambda: c.release(-1), lambda: c.release(2)):
        with pytest.raises(ValueError):
            call()
    assert c.share(0, 1, 0) == 0
    assert (c.table()[0] == -1).all() and (c.table()[1, :3] >= 0).all() and len(c._free) == 3


def test_refusals():
    with pytest.raises(ValueError):
        LatentCache(1, 0, 16, 64, device="cpu")
    c = LatentCache(2, 4, 16, 32, device="cpu")
    with pytest.raises(ValueError):
        c.reserve(0, 33)
    c.reserve(0, 16)
    with pytest.raises(ValueError):
        c.share(0, 1, 16)
    assert c.page_table.dtype == torch.int32


def test_a_capture_on_the_caches_own_device_is_what_counts(monkeypatch):
    """The check for a capture, and the upload, look at the cache's device and the
    call's stream, whichever device is the current one."""
    import contextlib
    at = []

    @contextlib.contextmanager
    def entered(name, what):
        at.append((name, what))
        yield
        at.pop()

    c = LatentCache(1, 4, 16, 64, device="cpu")
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered("device", d))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered("stream", s))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: ("device", torch.device("cuda:3")) in at)
    c.device = torch.device("cuda:3")
    c.reserve(0, 16)
    with pytest.raises(X.IdxError):
        c.table()
    assert (c.page_table == -1).all()                            # and the change is not forgotten
    c.device = torch.device("cpu")
    assert c.table()[0, 0] >= 0
