"""LatentCache's page table on its way to the device: an upload does not hold up
the host, carries the table as it was when the call was made, and is refused
inside a capture."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, UB, bf, tree_row

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,changed", [(64, 2), (64, 64)])
def test_upload_does_not_wait_for_the_stream(B, changed):
    """A few sequences have taken a page, or all of them: table() returns while
    the stream is still busy with earlier work, and later changes on the host do not
    reach an upload that has been asked for."""
    from sparse_attention_token_idx_b200.pipeline import LatentCache
    lc = LatentCache(B, 8 * B, 64, 512)
    for s in (None, torch.cuda.Stream()):
        st = s if s is not None else torch.cuda.current_stream()
        for b in range(B):
            lc.release(b)
            lc.reserve(b, 64)
        lc.table(s)
        for b in range(changed):                                 # staging memory of this size exists from here on
            lc.reserve(b, 128)
        lc.table(s)
        torch.cuda.synchronize()
        busy = torch.cuda.Event()
        with torch.cuda.stream(st):
            torch.cuda._sleep(400_000_000)                       # about 0.2 s
            busy.record(st)
        for b in range(changed):
            lc.reserve(b, 192)
        want = lc._table.clone()
        got = lc.table(s)
        held_up = busy.query()
        for b in range(B):
            lc.release(b)
        torch.cuda.synchronize()
        assert not held_up
        assert torch.equal(got.cpu(), want)
        assert bool((lc.table(s).cpu() == -1).all())


def test_a_changed_table_is_refused_inside_a_capture():
    from sparse_attention_token_idx_b200 import binding as X
    from sparse_attention_token_idx_b200.pipeline import LatentCache
    lc = LatentCache(2, 8, 64, 256)
    lc.reserve(0, 64)
    q = torch.zeros((2, 1, 16, DIM), dtype=torch.bfloat16, device="cuda")
    lens = dev(np.array([10, 0], np.int32))
    cnts = dev(np.array([1, 0], np.int32))
    out, lse = lc.attend(q, lens, 0.1, counts=cnts)              # loads the kernels, uploads the table
    torch.cuda.synchronize()
    lc.reserve(0, 128)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(X.IdxError):
            lc.attend(q, lens, 0.1, counts=cnts, out=out, lse=lse)
        with pytest.raises(X.IdxError):
            lc.table()
    lc.table()                                                   # still to be uploaded
    torch.cuda.synchronize()
    assert lc.page_table[0, 1].item() == lc._table[0, 1].item() >= 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lc.attend(q, lens, 0.1, counts=cnts, out=out, lse=lse)
    g.replay()
    torch.cuda.synchronize()
    assert X.status() == (0, 0)


def test_shared_prefix_then_rows_of_ones_own():
    """share(), append behind the shared rows, attend: both sequences read the
    prefix, each its own rows, and the prefix stays as it was."""
    from sparse_attention_token_idx_b200 import binding as X
    from sparse_attention_token_idx_b200.pipeline import LatentCache
    rng = np.random.default_rng(31)
    page, H, n = 16, 16, 5
    lc = LatentCache(2, 12, page, 128)
    gain = dev(np.ones(LAT, np.float32))
    one = lambda m: (torch.ones((2, m, 32), device="cuda"), torch.zeros((2, m, 32), device="cuda"))
    _, kv = bf(rng.standard_normal((2, 40, DIM)))
    lc.reserve(0, 40)
    lc.append(kv.cuda(), gain, 1e-6, *one(40), dev(np.zeros(2, np.int32)), counts=dev(np.array([40, 0], np.int32)))
    shared = lc.share(1, 0, 40)
    assert shared == 32
    before = lc.cache[lc._table[0, :2].long().cuda()].clone()
    starts = [40, shared]
    for b in range(2):
        lc.reserve(b, starts[b] + n)
    _, kv = bf(rng.standard_normal((2, n, DIM)))
    lc.append(kv.cuda(), gain, 1e-6, *one(n), dev(np.array(starts, np.int32)))
    assert torch.equal(lc.cache[lc._table[0, :2].long().cuda()], before)
    q64, q = bf(rng.standard_normal((2, n, H, DIM)))
    out, lse = lc.attend(q.cuda(), dev(np.array([s + n for s in starts], np.int32)), 0.07)
    assert X.status() == (0, 0)
    cache = lc.cache.double().cpu().numpy()
    for b in range(2):
        for i in range(n):
            t = np.arange(starts[b] + i + 1)
            kv = cache[lc._table[b].numpy()[t // page], t % page]
            o, ls, bound, lerr = tree_row(q64[b, i], kv, 0.07)
            assert np.all(np.abs(out[b, i].double().cpu().numpy() - o) <= bound + UB * np.abs(o) * (1 + UB) + 1e-30)
            assert np.all(np.abs(lse[b, i].double().cpu().numpy() - ls) <= lerr)


def test_calls_on_other_streams_come_behind_an_upload():
    """The upload is asked for on a busy stream; a call on another stream reads the
    table that it carries, and a second upload from there does not overtake it."""
    from sparse_attention_token_idx_b200.pipeline import LatentCache
    lc = LatentCache(4, 32, 64, 512)
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    for b in range(4):
        lc.reserve(b, 64)
    lc.table(busy)
    lc.reserve(0, 128)
    lc.table(other)                                              # (staging memory, kernels)
    copy = torch.zeros_like(lc.page_table)
    with torch.cuda.stream(other):
        copy.copy_(lc.page_table)
    torch.cuda.synchronize()
    lc.reserve(1, 192)
    want = lc._table.clone()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(200_000_000)                           # about 0.1 s
    lc.table(busy)
    with torch.cuda.stream(other):
        copy.copy_(lc.table())
    lc.reserve(2, 256)
    last = lc._table.clone()
    lc.table(other)
    torch.cuda.synchronize()
    assert torch.equal(copy.cpu(), want) and torch.equal(lc.page_table.cpu(), last)


def test_the_device_is_the_one_that_the_buffers_are_on():
    """"cuda" is a number from the start: later calls may be made with another
    device as the current one."""
    from sparse_attention_token_idx_b200.pipeline import Indexer, LatentCache
    now = torch.device("cuda", torch.cuda.current_device())
    assert LatentCache(1, 4, 16, 64).device == now
    assert Indexer(1, 64, 0, 8).device == now
