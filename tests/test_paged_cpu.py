"""Refusals of the paged latent cache's calls: the C entries' host checks (with
dummy addresses that are never dereferenced) and the Python wrappers' checks of
shapes, types and placement.  No GPU is touched."""
import pytest
import torch

P16 = 1 << 20            # a 16-byte aligned dummy address


def _append(lib, **kw):
    a = dict(kv=P16, kvs=576, kvt=576, gain=P16, eps=1e-6, cos=P16, sin=P16, inter=1, pos=P16, cnt=None, table=P16,
             max_pages=4, B=1, n=1, cache=P16, num_pages=8, page=64, q=P16, qs=64, qt=64, qh=64, H=16, qo=P16)
    a.update(kw)
    return lib.idx_latent_append(a["kv"], a["kvs"], a["kvt"], a["gain"], a["eps"], a["cos"], a["sin"], a["inter"],
                                 a["pos"], a["cnt"], a["table"], a["max_pages"], a["B"], a["n"], a["cache"],
                                 a["num_pages"], a["page"], a["q"], a["qs"], a["qt"], a["qh"], a["H"], a["qo"], None)


def _tree(lib, **kw):
    a = dict(q=P16, cache=P16, table=P16, max_pages=4, num_pages=8, page=64, L=P16, cnt=None, B=1, n=1, H=16,
             max_len=256, mask=None, idx=None, k=0, scale=0.1, out=P16, dt=1, lse=None, ws=P16, wsn=1 << 40)
    a.update(kw)
    return lib.idx_tree_mla(a["q"], a["cache"], a["table"], a["max_pages"], a["num_pages"], a["page"], a["L"], a["cnt"],
                            a["B"], a["n"], a["H"], a["max_len"], a["mask"], a["idx"], a["k"], a["scale"], a["out"],
                            a["dt"], a["lse"], a["ws"], a["wsn"], None)


SHAPE, NULL, FMT, K, ALIGN, SCRATCH = -2, -1, -3, -4, -5, -10


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), SHAPE), (dict(n=-1), SHAPE), (dict(H=-1), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(inter=2), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(page=0), SHAPE),
    (dict(num_pages=1 << 20, page=1 << 12), SHAPE), (dict(max_pages=1 << 20, page=1 << 12), SHAPE),
    (dict(B=0), 0), (dict(n=0, kv=None), 0),
    (dict(kv=None), NULL), (dict(gain=None), NULL), (dict(cos=None), NULL), (dict(pos=None), NULL),
    (dict(table=None), NULL), (dict(cache=None), NULL), (dict(q=None), NULL), (dict(qo=None), NULL),
    (dict(kv=P16 + 2), ALIGN), (dict(kvt=580), ALIGN), (dict(kvs=4), ALIGN), (dict(cache=P16 + 8), ALIGN),
    (dict(qh=68), ALIGN), (dict(qo=P16 + 8), ALIGN), (dict(gain=P16 + 4), ALIGN), (dict(sin=P16 + 8), ALIGN),
    (dict(B=1 << 30, n=1 << 10), SHAPE),
])
def test_append_host_checks(kw, code):
    from sparse_attention_token_idx_b200 import binding
    assert _append(binding.load(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), FMT), (dict(B=-1), SHAPE), (dict(n=65), SHAPE), (dict(H=0), SHAPE), (dict(k=-1), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(B=0), 0), (dict(n=0), 0),
    (dict(max_len=0), SHAPE), (dict(max_len=257), SHAPE), (dict(page=0), SHAPE), (dict(num_pages=0), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(num_pages=1 << 20, page=1 << 12), SHAPE),
    (dict(k=8), NULL), (dict(idx=P16), K),
    (dict(q=None), NULL), (dict(cache=None), NULL), (dict(table=None), NULL), (dict(L=None), NULL),
    (dict(out=None), NULL), (dict(q=P16 + 2), ALIGN), (dict(cache=P16 + 8), ALIGN), (dict(out=P16 + 8), ALIGN),
    (dict(ws=P16 + 8), ALIGN), (dict(mask=P16 + 4), ALIGN), (dict(B=1 << 24, n=64, H=1 << 20), SHAPE),
])
def test_tree_host_checks(kw, code):
    from sparse_attention_token_idx_b200 import binding
    assert _tree(binding.load(), **kw) == code


@pytest.mark.parametrize("scale,code", [(2.36e38, SHAPE), (-3.0e38, SHAPE), (2.3e38, NULL)])
def test_tree_refuses_a_scale_that_overflows_in_log2_units(scale, code):
    from sparse_attention_token_idx_b200 import binding
    assert _tree(binding.load(), scale=scale, q=None) == code      # (q = NULL: the next check)


def test_wrappers_reject_shapes_and_types_before_the_library():
    from sparse_attention_token_idx_b200 import binding as X
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = torch.zeros

    def tree(**kw):
        a = dict(q=z((2, 3, 16, 576), dtype=bf), cache=z((4, 64, 576), dtype=bf), page_table=z((2, 2), dtype=i32),
                 lengths=z(2, dtype=i32), softmax_scale=0.1, max_len=128)
        a.update(kw)
        return X.tree_mla(**a)

    for kw in (dict(q=z((2, 16, 576), dtype=bf)), dict(q=z((2, 3, 16, 512), dtype=bf)),
               dict(q=z((2, 65, 16, 576), dtype=bf)), dict(cache=z((4, 64, 512), dtype=bf)),
               dict(page_table=z((3, 2), dtype=i32)), dict(lengths=z(3, dtype=i32)), dict(counts=z(1, dtype=i32)),
               dict(tree_mask=z((2, 4), dtype=torch.int64)), dict(indices=z((2, 2, 8), dtype=i32)),
               dict(indices=z((2, 3, 0), dtype=i32)), dict(out=z((2, 3, 16, 576), dtype=bf)),
               dict(lse=z((2, 3), dtype=f32))):
        with pytest.raises(ValueError):
            tree(**kw)
    for kw in (dict(q=z((2, 3, 16, 576), dtype=f32)), dict(lengths=z(2, dtype=torch.int64)),
               dict(tree_mask=z((2, 3), dtype=i32)), dict(out=z((2, 3, 16, 512), dtype=torch.float16))):
        with pytest.raises(X.IdxError):
            tree(**kw)
    with pytest.raises(X.IdxError):
        tree()                                                   # CPU tensors

    def append(**kw):
        a = dict(kv_proj=z((2, 3, 576), dtype=bf), gain=z(512), eps=1e-6, rope_cos=z((2, 3, 32)),
                 rope_sin=z((2, 3, 32)), positions=z(2, dtype=i32), page_table=z((2, 2), dtype=i32),
                 cache=z((4, 64, 576), dtype=bf))
        a.update(kw)
        return X.latent_append(**a)

    for kw in (dict(kv_proj=z((2, 576), dtype=bf)), dict(kv_proj=z((2, 3, 640), dtype=bf)), dict(gain=z(576)),
               dict(rope_cos=z((2, 3, 64))), dict(positions=z(3, dtype=i32)), dict(page_table=z((1, 2), dtype=i32)),
               dict(q_pe=z((2, 3, 16, 128), dtype=bf)), dict(q_out=z((2, 3, 16, 576), dtype=bf)),
               dict(q_pe=z((2, 3, 16, 64), dtype=bf), q_out=z((2, 3, 8, 576), dtype=bf))):
        with pytest.raises(ValueError):
            append(**kw)
    for kw in (dict(gain=z(512, dtype=bf)), dict(positions=z(2, dtype=torch.int64)),
               dict(cache=z((4, 64, 576), dtype=f32))):
        with pytest.raises(X.IdxError):
            append(**kw)
    with pytest.raises(X.IdxError):
        append()                                                 # CPU tensors
