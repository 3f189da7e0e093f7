"""Shared by the tests of the paged latent cache: sequences laid out over a
randomly permuted page table, and both operators in float64 straight from their
definitions (numpy, one row at a time)."""
import numpy as np
import torch

LAT, ROT, DIM = 512, 64, 576
U = 2.0 ** -24          # half a step of fp32
UB = 2.0 ** -8          # half a step of bf16


def bf(x):
    """float array → the same values rounded to bf16, as (float64 values, bf16 CPU tensor)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t


class Paged:
    """B sequences of lens[b] rows over pages of `page` rows: a permuted page
    table (−1 past each sequence's end) and a cache filled with NaN where no
    sequence holds a row."""

    def __init__(self, rng, lens, page, extra=2, width=None):
        self.lens, self.page = list(lens), page
        need = [-(-x // page) for x in lens]
        self.width = width or max(1, max(need))
        self.num_pages = max(1, sum(need) + extra)
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.cache = np.full((self.num_pages, page, DIM), np.nan)

    def fill(self, rng, scale=1.0):
        for b, L in enumerate(self.lens):
            vals, _ = bf(scale * rng.standard_normal((L, DIM)))
            for t in range(L):
                self.cache[self.table[b, t // self.page], t % self.page] = vals[t]
        return self

    def rows(self, b, L):
        t = np.arange(L)
        return self.cache[self.table[b, t // self.page], t % self.page]

    def cache_dev(self):
        return torch.from_numpy(self.cache).to(torch.float32).to(torch.bfloat16).cuda()

    def table_dev(self):
        return torch.from_numpy(self.table).cuda()


def sees_draft(mask, b, i, j):
    return j <= i if mask is None else bool((int(mask[b][i]) >> j) & 1)


def row_positions(lens, cnts, mask, indices, b, i):
    ctx = lens[b] - cnts[b]
    if indices is None:
        pos = list(range(ctx))
    else:
        pos = [int(t) for t in indices[b, i] if 0 <= t < ctx]
    return pos + [ctx + j for j in range(cnts[b]) if sees_draft(mask, b, i, j)]


def tree_row(q, kv, scale):
    """One row's heads: q [H, 576], kv [m, 576] float64 → (out [H, 512], lse [H],
    bound factors): the output bound is rel·A + 2^-8·|out| (bf16 out), where
    A = Σ p |kv|; the lse bound is added as lse_err."""
    H = q.shape[0]
    if not len(kv):
        return np.zeros((H, LAT)), np.full(H, -np.inf), np.zeros((H, LAT)), np.zeros(H)
    s = scale * (q @ kv.T)
    # a score: 576 exact bf16 products summed in fp32, then two fp32 products by
    # the scale and log2 e (one rounding each, on the score's own size)
    e = (576 * U * abs(scale) * (np.abs(q) @ np.abs(kv).T) + 4 * U * np.abs(s)).max(axis=1)
    top = s.max(axis=1, keepdims=True)
    w = np.exp(s - top)
    z = w.sum(axis=1, keepdims=True)
    p = w / z
    # scores off by e move a weight by exp(±2e); exponentials (2^-22), sums,
    # rescalings and joins add (keys + 600)·2^-24; the bf16 weights 2^-8 each
    # above and below the division
    rel = np.expm1(2 * e) + (len(kv) + 600) * U + 2 * UB
    A = p @ np.abs(kv[:, :LAT])
    lse = (top + np.log(z))[:, 0]
    lse_err = e + (len(kv) + 600) * U + 4 * U * (np.abs(lse) + np.abs(top[:, 0]))
    return p @ kv[:, :LAT], lse, rel[:, None] * A, lse_err


def check_tree(got_out, got_lse, q, paged, cnts, scale, mask=None, indices=None, untouched=None):
    """Every row against its float64 value within the derived bound; rows behind
    the counts must hold `untouched`."""
    B, n = q.shape[:2]
    bf16_out = got_out.dtype == torch.bfloat16
    go, gl = got_out.double().cpu().numpy(), got_lse.double().cpu().numpy()
    for b in range(B):
        kvs = paged.rows(b, paged.lens[b])
        for i in range(n):
            if i >= cnts[b]:
                if untouched is not None:
                    assert np.all(go[b, i] == untouched) and np.all(gl[b, i] == untouched), (b, i)
                continue
            pos = row_positions(paged.lens, cnts, mask, indices, b, i)
            o, lse, bound, lse_err = tree_row(q[b, i], kvs[pos], scale)
            if not pos:
                assert np.all(go[b, i] == 0) and np.all(gl[b, i] == -np.inf), (b, i)
                continue
            bound = bound + (UB * np.abs(o) * (1 + UB) if bf16_out else 0) + 1e-30
            err = np.abs(go[b, i] - o)
            assert np.all(err <= bound), f"row {b},{i}: worst err/bound {np.nanmax(err / bound):.3f}"
            lerr = np.abs(gl[b, i] - lse)
            assert np.all(lerr <= lse_err), f"lse {b},{i}: worst {np.max(lerr / lse_err):.3f}"


def random_tree(rng, n):
    rows = []
    for i in range(n):
        par = -1 if i == 0 or rng.random() < 0.2 else int(rng.integers(max(0, i - 4), i))
        rows.append((1 << i) | (0 if par < 0 else rows[par]))
    return rows


def mask_dev(mask):
    return torch.tensor([[v - (1 << 64) if v >> 63 else v for v in row] for row in mask], dtype=torch.int64).cuda()
