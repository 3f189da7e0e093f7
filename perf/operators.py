"""Measured cases of the operators on the paged latent cache: the append of new
latent rows (norm and position rotation on the way), and the attention of
drafted token trees over the cache, dense or over an indexer's selection.

``run`` computes one pass of a case: with ``own`` false in elementary torch
operations (float32, rounded once at the end), with ``own`` true through the
library's calls.  ``exact`` computes the same outputs in float64.
"""
import math
import random

import torch

own = False

LAT, ROT, DIM = 512, 64, 576
EPS = 1e-6
NEG = float("-inf")


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one user's decode step on an eighth of the heads: one token, launch latency
        dict(name="append_one_token", op="append", B=1, n=1, H=16, page=64, ctx=1000, ragged=False, inter=True),
        # a full decode batch, all heads on this GPU (the batch of the decode benchmark)
        dict(name="append_decode_batch", op="append", B=128, n=1, H=128, page=64, ctx=16000, ragged=True, inter=True),
        # draft trees of different sizes in a padded batch, pages of 48 rows, half-split rotation
        dict(name="append_drafts_padded", op="append", B=37, n=13, H=16, page=48, ctx=3000, ragged=True, inter=False),
        # two prompt chunks of 2048 tokens (the chunked-prefill benchmark's shape)
        dict(name="append_prompt_chunk", op="append", B=2, n=2048, H=64, page=64, ctx=14336, ragged=False, inter=True),
        # one token over a short context: latency
        dict(name="tree_one_token_short", op="tree", B=1, n=1, H=16, page=64, ctx=150, ragged=False, k=0, mask="chain"),
        # plain decode over long ragged contexts on an eighth of the heads: the cache's bytes
        dict(name="tree_decode_long", op="tree", B=16, n=1, H=16, page=64, ctx=131000, ragged=True, k=0, mask="chain"),
        # trees of up to 13 drafts on an eighth of the heads, pages of 16 rows
        dict(name="tree_drafts_odd", op="tree", B=48, n=13, H=16, page=16, ctx=5001, ragged=True, k=0, mask="tree"),
        # trees of 8 drafts with all heads: the products
        dict(name="tree_drafts_full", op="tree", B=32, n=8, H=128, page=64, ctx=8192, ragged=True, k=0, mask="tree"),
        # two drafts over a small selection: latency
        dict(name="select_small", op="tree", B=1, n=2, H=16, page=64, ctx=1001, ragged=False, k=256, mask="chain"),
        # the decode benchmark's batch: 128 sequences of 16 384 positions, 2048 selected, all heads
        dict(name="select_decode_batch", op="tree", B=128, n=1, H=128, page=64, ctx=16383, ragged=False, k=2048,
             mask="chain"),
        # trees over selections, some contexts shorter than the selection, pages of 33 rows
        dict(name="select_drafts_odd", op="tree", B=16, n=7, H=16, page=33, ctx=9001, ragged=True, k=2048, mask="tree"),
        # short trees with all heads over selections
        dict(name="select_drafts_full", op="tree", B=64, n=4, H=128, page=64, ctx=16380, ragged=True, k=2048,
             mask="tree"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice([16, 32, 33, 48, 64, 100, 128])
    if rng.random() < 0.33:
        B, n = _log_int(rng, 1, 160), _log_int(rng, 1, 700)
        H = rng.choice([0, 1, 8, 16, 20, 64, 128])
        while B * n * max(H, 4) > 131072:
            n = max(1, n // 2)
            B = max(1, B - B // 4)
        return dict(op="append", B=B, n=n, H=H, page=page, ctx=_log_int(rng, 1, 20000), ragged=rng.random() < 0.6,
                    inter=rng.random() < 0.6)
    select = rng.random() < 0.5
    B, n, H = _log_int(rng, 1, 100), _log_int(rng, 1, 64 if not select else 16), rng.choice([1, 5, 8, 16, 24, 64, 128])
    ctx = _log_int(rng, 1, 100000)
    k = _log_int(rng, 1, 3000) if select else 0
    # at most the work of the largest listed case: rows × keys, and the rows read
    while B * n * H * (min(ctx, k) if select else ctx) > 120_000_000 or B * ctx > 1_800_000 or \
            (select and B * n * k > 500_000):
        if B > 1:
            B = max(1, B * 2 // 3)
        elif n > 1:
            n = max(1, n * 2 // 3)
        else:
            ctx = ctx * 2 // 3
    return dict(op="tree", B=B, n=n, H=H, page=page, ctx=max(1, ctx), ragged=rng.random() < 0.6, k=k,
                mask=rng.choice(["tree", "tree", "chain"]))


def _sizes(case):
    """(context lengths, new-token counts) of the case's sequences: fixed by the
    case, so that its work is.  Ragged batches hold a sequence without context."""
    B, n, ctx = case["B"], case["n"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B, [n] * B
    r = random.Random("%s %d %d %d %d" % (case["op"], B, n, ctx, case["page"]))
    ctxs = [int(ctx * (0.1 + 0.9 * r.random())) for _ in range(B)]
    cnts = [r.randint(max(1, n // 2), n) for _ in range(B)]
    ctxs[0], cnts[0] = ctx, n
    if B > 2:
        ctxs[1] = 0
    return ctxs, cnts


def _parents(case):
    """Parent of each draft (−1: a child of the context), one tree per sequence."""
    r = random.Random("tree %d %d %d" % (case["B"], case["n"], case["H"]))
    return [[-1 if i == 0 or r.random() < 0.15 else r.randint(max(0, i - 4), i - 1) for i in range(case["n"])]
            for _ in range(case["B"])]


def _mask_bits(case, cnts):
    """[B][n] bitmasks: bit j of row i is set where draft j is row i or one of its
    ancestors.  In ragged trees the last row of the second sequence (no context)
    sees nothing."""
    bits = []
    for b, par in enumerate(_parents(case)):
        rows = []
        for i in range(case["n"]):
            rows.append((1 << i) | (0 if par[i] < 0 else rows[par[i]]))
        if case["ragged"] and b == 1 and case["B"] > 2:
            rows[cnts[1] - 1] = 0
        bits.append(rows)
    return bits


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, n, H, page = case["B"], case["n"], case["H"], case["page"]
    ctxs, cnts = _sizes(case)
    lens = [c + m for c, m in zip(ctxs, cnts)]
    width = (max(lens) + page - 1) // page
    need = [(x + page - 1) // page for x in lens]
    pages = sum(need) + 3
    dev = dict(device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    st = dict(op=case["op"], B=B, n=n, H=H, page=page)
    # pages handed out in a random order; table entries past a sequence's end are −1
    order = torch.randperm(pages, generator=g, **dev).to(torch.int32)
    starts = torch.tensor([sum(need[:b]) for b in range(B)], **dev)
    col = torch.arange(width, **dev)
    held = col[None, :] < torch.tensor(need, **dev)[:, None]
    at = (starts[:, None] + col[None, :]).clamp(max=pages - 1)
    st["table"] = torch.where(held, order[at], torch.full((), -1, **i32)).contiguous()
    st["lengths"] = torch.tensor(lens, **i32)
    st["counts"] = torch.tensor(cnts, **i32) if case["ragged"] else None

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if case["op"] == "append":
        st["cache"] = torch.zeros((pages, page, DIM), dtype=torch.bfloat16, **dev)
        # the key projection is the tail of a wider fused projection: strided rows
        st["kv"] = (normal(B, n, 192 + DIM) * 1.7)[..., 192:]
        st["gain"] = 1 + 0.2 * torch.randn(LAT, generator=g, **dev)
        ctx = torch.tensor(ctxs, **dev)
        # a draft's position is its depth after the context; its slot is its index
        depth = torch.tensor([[i - (i % 3 if n <= 64 else 0) for i in range(n)]], **dev)
        freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, **dev) / 32)
        ang = (ctx[:, None] + depth).double()[..., None] * freq
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        st["positions"] = torch.tensor(ctxs, **i32)
        st["inter"] = case["inter"]
        st["q_pe"] = normal(B, n, H, 192)[..., 128:] if H else None
        st["q"] = normal(B, n, H, DIM) if H else None
        return st

    st["cache"] = normal(pages, page, DIM)
    # rows that no sequence holds are whatever memory held: not numbers
    tail = [b for b in range(B) if lens[b] % page]
    if tail:
        last = st["table"].long()[tail, [need[b] - 1 for b in tail]]
        gone = torch.arange(page, **dev)[None, :] >= torch.tensor([lens[b] % page for b in tail], **dev)[:, None]
        st["cache"][last] = torch.where(gone[..., None], float("nan"), st["cache"][last])
    st["q"] = normal(B, n, H, DIM)
    st["scale"] = 192 ** -0.5
    st["max_len"] = max(lens)
    st["mask"] = None
    if case["mask"] == "tree":
        two = [[v - (1 << 64) if v >> 63 else v for v in row] for row in _mask_bits(case, cnts)]
        st["mask"] = torch.tensor(two, dtype=torch.int64, **dev)
    st["idx"] = None
    if case["k"]:
        # what an indexer returns: distinct positions of the context, −1 behind them
        k, m = case["k"], max(1, max(ctxs))
        ctx = torch.tensor(ctxs, **dev)
        rnd = torch.rand((B, n, m), generator=g, **dev)
        rnd = torch.where(torch.arange(m, **dev) < ctx[:, None, None], rnd, -1.0)
        top = rnd.topk(min(k, m), dim=-1)
        idx = torch.full((B, n, k), -1, **i32)
        idx[..., :top.indices.shape[-1]] = torch.where(top.values >= 0, top.indices, -1).to(torch.int32)
        st["idx"] = idx
    # static output buffers, as a decode loop keeps them: rows behind a sequence's
    # last draft are left as they were
    st["out"] = torch.zeros((B, n, H, LAT), dtype=torch.bfloat16, **dev)
    st["lse"] = torch.zeros((B, n, H), dtype=torch.float32, **dev)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        from sparse_attention_token_idx_b200 import binding as X
        if st["op"] == "append":
            X.latent_append(st["kv"], st["gain"], EPS, st["cos"], st["sin"], st["positions"], st["table"], st["cache"],
                            interleaved=st["inter"], counts=st["counts"], q_pe=st["q_pe"], q_out=st["q"])
            return {"cache": st["cache"]} if st["q"] is None else {"cache": st["cache"], "q": st["q"]}
        out, lse = X.tree_mla(st["q"], st["cache"], st["table"], st["lengths"], st["scale"], max_len=st["max_len"],
                              counts=st["counts"], tree_mask=st["mask"], indices=st["idx"], out=st["out"],
                              lse=st["lse"])
        return {"out": out, "lse": lse}
    if st["op"] == "append":
        return _plain_append(st)
    return _plain_tree(st)


def _plain_rotate(x, cos, sin, inter):
    """The 64 rotary features of x, turned by the angles' cosines and sines."""
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :32], x[..., 32:])
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)


def _plain_append(st):
    B, n, page = st["B"], st["n"], st["page"]
    x = st["kv"].float()
    lat = x[..., :LAT]
    lat = lat * (1 / torch.sqrt((lat * lat).mean(-1, keepdim=True) + EPS)) * st["gain"]
    rot = _plain_rotate(x[..., LAT:], st["cos"], st["sin"], st["inter"])
    row = torch.cat((lat, rot), -1).to(torch.bfloat16)
    i = torch.arange(n, device=row.device)
    cnt = st["counts"] if st["counts"] is not None else torch.full_like(st["lengths"], n)
    real = i[None, :] < cnt[:, None]
    slot = (st["positions"][:, None] + i).long()
    slot = torch.where(real, slot, 0)
    where = st["table"].long().gather(1, slot // page).clamp(min=0) * page + slot % page
    st["cache"].view(-1, DIM)[where[real]] = row[real]
    if st["q"] is None:
        return {"cache": st["cache"]}
    rot = _plain_rotate(st["q_pe"].float(), st["cos"][:, :, None], st["sin"][:, :, None], st["inter"])
    st["q"][..., LAT:] = torch.where(real[..., None, None], rot.to(torch.bfloat16), st["q"][..., LAT:])
    return {"cache": st["cache"], "q": st["q"]}


def _plain_tree(st):
    B, n, H, page = st["B"], st["n"], st["H"], st["page"]
    dev = st["q"].device
    cnt = st["counts"].long() if st["counts"] is not None else torch.full((B,), n, device=dev)
    ctx = st["lengths"].long() - cnt
    i = torch.arange(n, device=dev)
    if st["mask"] is None:
        sees = (i[None, :] <= i[:, None])[None].expand(B, n, n)
    else:
        sees = (st["mask"][..., None] >> i) & 1 != 0
    sees = sees & (i < cnt[:, None])[:, None, :]                       # [B, row, draft]
    drafts = (ctx[:, None] + i)[:, None, :].expand(B, n, n)
    flat = st["cache"].view(-1, DIM)
    if st["idx"] is not None:                                          # keys of each row: its selection, its drafts
        sel = st["idx"].long()
        slot = torch.cat((sel, drafts), -1)
        seen = torch.cat(((sel >= 0) & (sel < ctx[:, None, None]), sees), -1)
        slot = torch.where(seen, slot, 0)
        table = st["table"].long()[:, None, :].expand(B, n, -1)
        kv = flat[table.gather(2, slot // page).clamp(min=0) * page + slot % page]
        kv = torch.where(seen[..., None], kv, 0).float()               # [B, n, keys, 576]
        s = torch.einsum("bihd,bikd->bihk", st["q"].float(), kv) * st["scale"]
        s = torch.where(seen[:, :, None, :], s, NEG)
    else:                                                              # keys of each sequence: its whole cache
        L = st["max_len"]
        t = torch.arange(L, device=dev)
        slot = torch.where(t < st["lengths"][:, None], t, 0)
        kv = flat[st["table"].long().gather(1, slot // page).clamp(min=0) * page + slot % page]
        kv = torch.where((t < st["lengths"][:, None])[..., None], kv, 0).float()   # [B, L, 576]
        d = t[None, :] - ctx[:, None]                                  # draft number of each slot
        seen = (d < 0)[:, None, :] | ((d >= 0) & (d < n))[:, None, :] & \
            sees.gather(2, d.clamp(0, n - 1)[:, None, :].expand(B, n, L))
        s = torch.einsum("bihd,bkd->bihk", st["q"].float(), kv) * st["scale"]
        s = torch.where(seen[:, :, None, :], s, NEG)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == NEG, 0, top))
    z = e.sum(-1, keepdim=True)
    v = kv[..., :LAT]
    o = torch.einsum("bihk,bikd->bihd" if st["idx"] is not None else "bihk,bkd->bihd", e, v) / torch.where(z == 0, 1, z)
    lse = (top + torch.log(z))[..., 0]
    real = (i[None, :] < cnt[:, None])[:, :, None]
    return {"out": torch.where(real[..., None], o.to(torch.bfloat16), 0), "lse": torch.where(real, lse, 0.0)}


# ---------------------------------------------------------------- the floor
def work(case):
    B, n, H = case["B"], case["n"], case["H"]
    ctxs, cnts = _sizes(case)
    tokens = sum(cnts)
    if case["op"] == "append":
        return {"bytes": tokens * (DIM * 2 * 2 + H * ROT * 2 * 2 + 2 * 32 * 4) + LAT * 4,
                "flops": tokens * (LAT * 4 + (1 + H) * ROT * 3)}
    keys = products = 0
    for b in range(B):
        if case["k"]:
            per = min(case["k"], ctxs[b])
            keys += min(ctxs[b], per * cnts[b]) + cnts[b]
            products += cnts[b] * (per + (cnts[b] + 1) // 2)
        else:
            keys += ctxs[b] + cnts[b]
            products += cnts[b] * (ctxs[b] + (cnts[b] + 1) // 2)
    return {"bytes": keys * DIM * 2 + tokens * H * (DIM * 2 + LAT * 2 + 4) + (tokens * case["k"] * 4),
            "flops": products * H * 2 * (DIM + LAT)}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, st)
    ctxs, cnts = _sizes(case)
    if work(case)["flops"] > 6e12:
        return None
    B, n, H, page = case["B"], case["n"], case["H"], case["page"]
    out = torch.zeros((B, n, H, LAT), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, n, H), dtype=torch.float64, device="cuda")
    bits = _mask_bits(case, cnts) if case["mask"] == "tree" else [[(2 << i) - 1 for i in range(n)]] * B
    for b in range(B):
        rows = (ctxs[b] + cnts[b] + page - 1) // page
        seq = st["cache"][st["table"][b, :rows].long()].reshape(-1, DIM)[:ctxs[b] + cnts[b]].double()
        before = ctxs[b]
        for i in range(cnts[b]):
            mine = [before + j for j in range(cnts[b]) if bits[b][i] >> j & 1]
            mine = torch.tensor(mine, dtype=torch.int64, device="cuda")
            if case["k"]:
                sel = st["idx"][b, i].long()
                kv = seq[torch.cat((sel[sel >= 0], mine))]
            else:
                kv = torch.cat((seq[:before], seq[mine])) if before else seq[mine]
            if not kv.shape[0]:
                lse[b, i] = NEG
                continue
            s = st["q"][b, i].double() @ kv.T * 192 ** -0.5
            lse[b, i] = torch.logsumexp(s, 1)
            out[b, i] = torch.exp(s - lse[b, i][:, None]) @ kv[:, :LAT]
    return {"out": out, "lse": lse}


def _exact_append(case, st):
    ctxs, cnts = _sizes(case)
    cache, page = st["cache"].double(), case["page"]
    c, s = st["cos"].double(), st["sin"].double()

    def turn(x, c, s):
        z = torch.complex(x[..., 0::2], x[..., 1::2]) if case["inter"] else torch.complex(x[..., :32], x[..., 32:])
        z = z * torch.complex(c, s)
        y = torch.view_as_real(z)
        return y.reshape(x.shape) if case["inter"] else torch.cat((y[..., 0], y[..., 1]), -1)

    for b in range(case["B"]):
        x = st["kv"][b, :cnts[b]].double()
        lat = x[:, :LAT] / torch.sqrt(x[:, :LAT].pow(2).sum(1, keepdim=True) / LAT + EPS) * st["gain"].double()
        new = torch.cat((lat, turn(x[:, LAT:], c[b, :cnts[b]], s[b, :cnts[b]])), 1)
        slots = torch.arange(ctxs[b], ctxs[b] + cnts[b], device="cuda")
        cache[st["table"][b].long()[slots // page], slots % page] = new
    if not case["H"]:
        return {"cache": cache}
    q = st["q"].double()
    for b in range(case["B"]):
        m = cnts[b]
        q[b, :m, :, LAT:] = turn(st["q_pe"][b, :m].double(), c[b, :m, None], s[b, :m, None])
    return {"cache": cache, "q": q}
