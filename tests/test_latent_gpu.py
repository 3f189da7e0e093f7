"""Append to the paged latent cache (idx_latent_append) against float64.

Bounds: a latent feature is x·r·g with r from a 512-term fp32 sum of squares: the
sum is off by at most 512·2^-24 relative, its root by half that, plus a few
roundings: 300·2^-24 in all, then half a bf16 step, 2^-8.  A rotated feature is
off by 3·2^-24·(|a cos| + |b sin|), then half a bf16 step."""
import numpy as np
import pytest
import torch

from tests.helpers import dev
from tests.paged_helpers import DIM, LAT, ROT, U, UB, Paged, bf

pytestmark = pytest.mark.gpu


def _turn(x, c, s, inter):
    """Rotation of the last 64 features (float64) and the size its errors scale with."""
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, a * s + b * c
    mu, mv = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    if inter:
        return np.stack((u, v), -1).reshape(x.shape), np.stack((mu, mv), -1).reshape(x.shape)
    return np.concatenate((u, v), -1), np.concatenate((mu, mv), -1)


def _inputs(rng, B, n, H, pad_kv=0, head=ROT):
    kv64, kv = bf(1.5 * rng.standard_normal((B, n, pad_kv + DIM)))
    gain = (1 + 0.3 * rng.standard_normal(LAT)).astype(np.float32)
    ang = rng.uniform(-400, 400, (B, n, ROT // 2))
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    q64, q = bf(rng.standard_normal((B, n, max(H, 1), head)))
    return kv64[..., pad_kv:], kv.cuda()[..., pad_kv:], gain, c, s, q64[..., head - ROT:], q.cuda()[..., head - ROT:]


@pytest.mark.parametrize("B,n,H,page,starts,cnts,inter,pad_kv,head", [
    (1, 1, 16, 64, [0], None, True, 0, 64),                     # the first token of a sequence
    (1, 1, 1, 1, [5], None, False, 8, 64),                      # one head, pages of one row
    (3, 5, 20, 33, [0, 31, 64], [5, 0, 3], True, 192, 192),     # ragged, one sequence without new tokens
    (2, 70, 7, 48, [40, 0], [70, 1], False, 64, 192),           # pages end inside the run
    (4, 3, 128, 16, [15, 16, 17, 1000], None, True, 1536, 192),
    (2, 9, 0, 100, [99, 7], [9, 8], False, 0, 64),              # keys only
])
def test_append_matches_float64(B, n, H, page, starts, cnts, inter, pad_kv, head):
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(B * 1000 + n * 10 + H)
    real = cnts or [n] * B
    kv64, kv, gain, c, s, q64, q = _inputs(rng, B, n, H, pad_kv, head)
    paged = Paged(rng, [a + m for a, m in zip(starts, real)], page)
    eps = 1e-6
    cache = torch.full((paged.num_pages, page, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = torch.full((B, n, H, DIM), -3.0, dtype=torch.bfloat16, device="cuda") if H else None
    X.latent_append(kv, dev(gain), eps, dev(c), dev(s), dev(np.array(starts, np.int32)), paged.table_dev(), cache,
                    interleaved=inter, counts=dev(np.array(cnts, np.int32)) if cnts else None, q_pe=q if H else None,
                    q_out=q_out)
    assert X.status() == (0, 0)
    got = cache.double().cpu().numpy()
    c64, s64 = c.astype(np.float64), s.astype(np.float64)
    written = np.zeros((paged.num_pages, page), bool)
    for b in range(B):
        for i in range(real[b]):
            x = kv64[b, i]
            lat = x[:LAT] / np.sqrt(np.mean(x[:LAT] ** 2) + eps) * gain
            rot, size = _turn(x[LAT:], c64[b, i], s64[b, i], inter)
            ref = np.concatenate((lat, rot))
            bound = np.concatenate((np.abs(lat) * (UB + 300 * U * (1 + UB)),
                                    UB * np.abs(rot) + 3 * U * size * (1 + UB))) + 1e-38
            t = starts[b] + i
            pg, r = paged.table[b, t // page], t % page
            written[pg, r] = True
            assert np.all(np.abs(got[pg, r] - ref) <= bound), (b, i)
    assert np.all(got[~written] == 7.0)                          # every other row as it was
    if H:
        gq = q_out.double().cpu().numpy()
        assert np.all(gq[..., :LAT] == -3.0)
        for b in range(B):
            assert np.all(gq[b, real[b]:] == -3.0)
            rot, size = _turn(q64[b], c64[b][:, None], s64[b][:, None], inter)
            bound = UB * np.abs(rot) + 3 * U * size * (1 + UB) + 1e-38
            m = real[b]
            assert np.all(np.abs(gq[b, :m, :, LAT:] - rot[:m]) <= bound[:m])


def test_rotation_in_place_of_the_joined_query():
    """q_pe may be the rotary part of q_out itself."""
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(3)
    B, n, H = 2, 3, 24
    kv64, kv, gain, c, s, _, _ = _inputs(rng, B, n, H)
    _, qj = bf(rng.standard_normal((B, n, H, DIM)))
    for inter in (True, False):
        want, q = torch.zeros((B, n, H, DIM), dtype=torch.bfloat16, device="cuda"), qj.cuda()
        args = (kv, dev(gain), 1e-6, dev(c), dev(s), dev(np.zeros(B, np.int32)), dev(np.array([[0], [1]], np.int32)),
                torch.zeros((2, 8, DIM), dtype=torch.bfloat16, device="cuda"))
        X.latent_append(*args, interleaved=inter, q_pe=q[..., LAT:].clone(), q_out=want)
        X.latent_append(*args, interleaved=inter, q_pe=q[..., LAT:], q_out=q)
        assert torch.equal(q[..., LAT:], want[..., LAT:]) and torch.equal(q[..., :LAT], qj.cuda()[..., :LAT])


def test_errors_that_depend_on_data_write_nothing():
    from sparse_attention_token_idx_b200 import binding as X
    rng = np.random.default_rng(4)
    B, n, H, page = 4, 2, 16, 8
    kv64, kv, gain, c, s, q64, q = _inputs(rng, B, n, H)
    table = dev(np.array([[0, 1], [2, 3], [4, 99], [6, 7]], np.int32))

    def go(starts, cnts):
        cache = torch.zeros((8, page, DIM), dtype=torch.bfloat16, device="cuda")
        qo = torch.zeros((B, n, H, DIM), dtype=torch.bfloat16, device="cuda")
        X.latent_append(kv, dev(gain), 1e-6, dev(c), dev(s), dev(np.array(starts, np.int32)), table, cache,
                        counts=dev(np.array(cnts, np.int32)), q_pe=q, q_out=qo)
        code, bits = X.status()
        held = cache.abs().sum(-1).ne(0).nonzero().cpu().numpy().tolist()
        return code, bits, held, [b for b in range(B) if qo[b].abs().sum().item()]

    assert go([0, 0, 0, 0], [2, 2, 2, 2])[:2] == (0, 0)
    code, bits, held, qs = go([-1, 15, 0, 0], [2, 2, 2, 2])      # before the first slot; past the last
    assert code == -7 and bits == X.DEV_ERR_POSITION and held == [[4, 0], [4, 1], [6, 0], [6, 1]] and qs == [2, 3]
    code, bits, held, qs = go([0, 0, 0, 0], [3, -1, 1, 0])       # counts outside [0, n]
    assert code == -7 and bits == X.DEV_ERR_LENGTH and held == [[4, 0]] and qs == [2]
    code, bits, held, qs = go([0, 0, 7, 0], [0, 0, 2, 0])        # the second token's page is no page
    assert code == -7 and bits == X.DEV_ERR_PAGE and held == [[4, 7]] and qs == [2]
    assert X.status() == (0, 0)
