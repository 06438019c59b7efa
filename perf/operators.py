"""Timed cases of the latent-cache operators: the step's tables, the cache
write, the attention that reads the cache (dense or drafted-tree over pages,
over selected rows, and expanded per head for prompts) and the join of ranks.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare(case, seed)` makes one case's inputs on the GPU, `run(state)` makes
one pass: in plain torch operations, or through the package where `own` is
true.  `work(case)` counts what a pass cannot do without, and
`exact(case, seed)` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # a decode step: one new token for each running request of one rank in eight
        dict(name="tables_decode", op="tables", requests=32, new=1, context=65536, block=64,
             ranks=8, drafted=False),
        # a mixed step of a large batch: prompts' chunks next to single tokens
        dict(name="tables_mixed", op="tables", requests=1024, new=64, context=16384, block=64,
             ranks=1, drafted=False),
        # a decode step's cache write
        dict(name="store_decode", op="store", tokens=32, latent=384, tail=64, dtype="bf16",
             interleaved=False),
        # a prompt chunk's cache write
        dict(name="store_chunk", op="store", tokens=16384, latent=512, tail=32, dtype="bf16",
             interleaved=True),
        # decode over whole contexts of ragged length, one token a request
        dict(name="paged_decode", op="attend", requests=64, new=1, context=16384, heads=32,
             latent=384, tail=64, block=64, tree=False, dtype="bf16"),
        # verification of drafted trees, small pages, an odd context
        dict(name="paged_tree", op="attend", requests=4, new=24, context=6001, heads=16,
             latent=256, tail=32, block=16, tree=True, dtype="fp16"),
        # one token over its selected rows: the smallest call of a decode step
        dict(name="rows_single", op="rows", requests=1, new=1, context=8192, k=512, heads=20,
             latent=256, tail=64, block=64, dtype="bf16"),
        # the decode merge's batch over its selected rows
        dict(name="rows_decode", op="rows", requests=128, new=1, context=16384, k=2048,
             heads=64, latent=512, tail=32, block=64, dtype="bf16"),
        # a few ragged prompts, none with a context
        dict(name="expanded_prompts", op="expanded", requests=5, new=391, context=0, heads=12,
             nope=64, tail=32, value=64, dtype="fp16"),
        # a prompt chunk of 4096 tokens whose keys are 8192 columns
        dict(name="expanded_chunk", op="expanded", requests=1, new=4096, context=4096, heads=16,
             nope=128, tail=64, value=128, dtype="bf16"),
        # two ranks' partial results of a small step
        dict(name="merge_small", op="merge", ranks=2, tokens=8, heads=16, latent=256,
             dtype="bf16"),
        # eight ranks' partial results of the decode merge's batch
        dict(name="merge_decode", op="merge", ranks=8, tokens=128, heads=64, latent=512,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_one(rng):
    op = rng.choice(["tables", "store", "attend", "attend", "rows", "rows", "expanded", "merge"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    latent = 16 * _log_int(rng, 2, 32)
    tail = rng.choice([0, 16, 32, 48, 64])
    block = rng.choice([16, 32, 64, 128])
    if op == "tables":
        return dict(op=op, requests=_log_int(rng, 1, 1024), new=_log_int(rng, 1, 64),
                    context=_log_int(rng, 16, 65536), block=block, ranks=rng.choice([1, 1, 2, 8]),
                    drafted=rng.random() < 0.3)
    if op == "store":
        return dict(op=op, tokens=_log_int(rng, 1, 16384), latent=latent, tail=tail, dtype=dtype,
                    interleaved=rng.random() < 0.5)
    if op == "attend":
        new = rng.choice([1, 1, _log_int(rng, 2, 48)])
        return dict(op=op, requests=_log_int(rng, 1, 64), new=new,
                    context=_log_int(rng, 8, 16384), heads=_log_int(rng, 1, 128), latent=latent,
                    tail=tail, block=block, tree=new > 1 and rng.random() < 0.6, dtype=dtype)
    if op == "rows":
        return dict(op=op, requests=_log_int(rng, 1, 128), new=rng.choice([1, 1, 4, 7]),
                    context=_log_int(rng, 64, 16384), k=_log_int(rng, 16, 2048),
                    heads=_log_int(rng, 1, 128), latent=latent, tail=tail, block=block,
                    dtype=dtype)
    if op == "expanded":
        return dict(op=op, requests=_log_int(rng, 1, 12), new=_log_int(rng, 1, 4096),
                    context=rng.choice([0, _log_int(rng, 1, 4096)]), heads=_log_int(rng, 1, 32),
                    nope=16 * rng.randint(2, 8), tail=tail, value=16 * rng.randint(2, 8),
                    dtype=dtype)
    return dict(op=op, ranks=rng.randint(2, 8), tokens=_log_int(rng, 1, 128),
                heads=_log_int(rng, 1, 128), latent=latent, dtype=dtype)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw_one(rng)
        if _cost(c) <= most[c["op"]]:
            return c


# --- what a case's seed does not change ------------------------------------

def _context_lens(case):
    """Cached tokens of each request before the step: ragged, a quarter to the
    whole of `context`; from four requests on, one has an empty cache."""
    R, L = case["requests"], case["context"]
    lens = np.linspace(L, L / 4, R).astype(np.int64)
    if R >= 4:
        lens[1] = 0
    return lens


def _new_lens(case):
    """New tokens of each request: the case's `new` and below, one at least."""
    R, n = case["requests"], case["new"]
    return np.maximum(1, np.linspace(n, max(1, n // 3), R).astype(np.int64))


def _rows_counts(case):
    """Selected rows of each token: k, or fewer for every fifth token and where
    the context is shorter than k."""
    T = case["requests"] * case["new"]
    n = min(case["k"], case["context"])
    return np.where(np.arange(T) % 5 == 4, n - n // 3, n)


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    op = case["op"]
    if op == "tables":
        R = case["requests"]
        T = int(_new_lens(case).sum())
        c, n, W, B = _context_lens(case), _new_lens(case), case["ranks"], case["block"]
        blocks = int((_cdiv((c + n + W - 1) // W, B) - _cdiv((c + W - 1) // W, B)).sum())
        # lengths in, per-token and per-request arrays out, new blocks through,
        # the table entry of each token's block in
        return {"bytes": 8 * R + 16 * T + 8 * R + 8 * blocks + 4 * R, "flops": 0}
    if op == "store":
        T, D = case["tokens"], case["latent"] + case["tail"]
        rope = case["tail"] * 4 if case["tail"] else 0
        return {"bytes": T * (4 * D + rope + 8) + 4 * case["latent"],
                "flops": T * (4 * case["latent"] + 3 * case["tail"])}
    if op == "attend":
        R, n, H = case["requests"], case["new"], case["heads"]
        D = case["latent"] + case["tail"]
        base = _context_lens(case)
        keys = base + n if case["tree"] or n > 1 else base
        pairs = sum(n * int(b) + (n * (n + 1) // 2 if n > 1 else 0) for b in base)
        io = R * n * H * ((D + case["latent"]) * 2 + 4)
        return {"bytes": int(keys.sum()) * D * 2 + io, "flops": 2 * pairs * H * (D + case["latent"])}
    if op == "rows":
        H, D = case["heads"], case["latent"] + case["tail"]
        counts = _rows_counts(case)
        T = len(counts)
        n = case["new"]
        distinct = sum(min(int(counts[r * n:(r + 1) * n].sum()), case["context"])
                       for r in range(case["requests"]))
        io = T * H * ((D + case["latent"]) * 2 + 4) + 4 * int(counts.sum())
        return {"bytes": distinct * D * 2 + io,
                "flops": 2 * int(counts.sum()) * H * (D + case["latent"])}
    if op == "expanded":
        H, D, dv = case["heads"], case["nope"] + case["tail"], case["value"]
        n, c = _new_lens(case), np.full(case["requests"], case["context"])
        T, S = int(n.sum()), int((n + c).sum())
        pairs = int((n * c + n * (n + 1) // 2).sum())
        return {"bytes": T * H * ((D + dv) * 2 + 4) + S * (H * (case["nope"] + dv) + case["tail"]) * 2,
                "flops": 2 * pairs * H * (D + dv)}
    n = case["tokens"] * case["heads"]
    per = case["latent"] * 2 + 4
    return {"bytes": n * per * (case["ranks"] + 1), "flops": 2 * n * case["latent"] * case["ranks"]}


# --- inputs -----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, offset=None):
    """Standard normal values of `dtype`, on top of an offset shared by all rows
    (cached vectors of a model share a direction)."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    x.normal_(generator=g)
    if offset is not None:
        x.add_(offset.to(dtype))
    return x


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _pages(rng, requests, keys, block):
    """A pool of blocks handed out in random order: int32 [requests, width]."""
    width = max(1, _cdiv(keys, block))
    ids = rng.permutation(requests * width + 3)[:requests * width]
    return ids.reshape(requests, width), (requests * width + 3) * block


def _tree_words(rng, requests, n):
    """Ancestor bits of random trees of n drafted tokens, each token's own bit
    among them: int32 [requests * n, words]."""
    words = _cdiv(n, 32)
    out = np.zeros((requests * n, words), dtype=np.uint32)
    for r in range(requests):
        for i in range(n):
            row = out[r * n + i]
            if i and (i < 3 or rng.random() < 0.8):
                row |= out[r * n + rng.randint(max(0, i - 6), i)]
            row[i // 32] |= np.uint32(1 << (i % 32))
    return out.view(np.int32)


def prepare(case, seed):
    op = case["op"]
    rng = np.random.RandomState(seed % (1 << 32))
    g = _gen(seed)
    dt = DTYPES[case["dtype"]] if "dtype" in case else None
    s = dict(case=case)
    if op == "tables":
        R, B, W = case["requests"], case["block"], case["ranks"]
        perm = rng.permutation(R)
        ctx, new = _context_lens(case)[perm], _new_lens(case)[rng.permutation(R)]
        if case["context"] > 64:  # contexts end anywhere in a block
            ctx = np.maximum(0, ctx - rng.randint(0, 64, R))
        width = _cdiv(_cdiv(case["context"] + case["new"], W), B) + 1
        blocks = rng.permutation(2 * R * width)
        table = np.where(np.arange(width)[None] < _cdiv((ctx + W - 1) // W, B)[:, None],
                         blocks[:R * width].reshape(R, width), -1)
        s.update(context=_i32(ctx), new=_i32(new), table=_i32(table), rank=int(rng.randint(W)),
                 free=_i32(blocks[R * width:]),
                 tokens=int(new.sum()) + 3)  # three spare entries
    elif op == "store":
        T, dl, dr = case["tokens"], case["latent"], case["tail"]
        rows = 2 * T + 5
        P = 16384
        inv = 10000.0 ** (-torch.arange(0, max(dr, 2), 2, dtype=torch.float64) / max(dr, 2))
        ang = torch.arange(P, dtype=torch.float64)[:, None] * inv
        s.update(latent=_normal(g, (T, dl), dt).mul_(3), tail=_normal(g, (T, dr), dt),
                 weight=torch.rand(dl, generator=g, device=DEV) + 0.5,
                 cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)[:, :max(dr, 1)],
                 positions=_i32(rng.randint(0, P, T)), slots=_i32(rng.permutation(rows)[:T]),
                 cache=torch.zeros(rows, dl + dr, dtype=dt, device=DEV))
        s["slots"][::7] = -1  # tokens that another rank holds
        if T == 1:
            s["slots"][0] = 1
    elif op in ("attend", "rows"):
        R, n, L, H = case["requests"], case["new"], case["context"], case["heads"]
        dl, D, B = case["latent"], case["latent"] + case["tail"], case["block"]
        keys = L + (n if op == "attend" else 0)
        table, rows = _pages(rng, R, keys, B)
        off = 0.5 * torch.randn(D, generator=g, device=DEV)
        s.update(q=_normal(g, (R * n, H, D), dt), cache=_normal(g, (rows, D), dt, off),
                 scale=1.25 / math.sqrt(D))
        if op == "attend":
            base = _context_lens(case)[rng.permutation(R)]
            ends = np.repeat(base, n)
            if not case["tree"] and n > 1:  # a chunk: each token sees those before it
                ends = ends + np.tile(np.arange(1, n + 1), R)
            s.update(table=_i32(table), ends=_i32(ends), req=_i32(np.repeat(np.arange(R), n)),
                     tree=torch.from_numpy(_tree_words(rng, R, n)).to(DEV) if case["tree"] else None)
        else:
            k = case["k"]
            counts = _i32(_rows_counts(case))
            pick = torch.rand(R * n, L, generator=g, device=DEV).topk(min(k, L), dim=1).indices
            pick = pick.sort(dim=1).values
            t = _i32(table).long().repeat_interleave(n, 0)
            phys = t.gather(1, pick // B) * B + pick % B
            out = torch.full((R * n, k), -1, dtype=torch.int32, device=DEV)
            out[:, :phys.shape[1]] = phys.int()
            out[torch.arange(k, device=DEV)[None] >= counts[:, None]] = -1
            s.update(rows=out, counts=counts)
    elif op == "expanded":
        H, dn, dr, dv = case["heads"], case["nope"], case["tail"], case["value"]
        new = _new_lens(case)[rng.permutation(case["requests"])]
        klen = new + case["context"]
        T, S = int(new.sum()), int(klen.sum())
        ends = np.concatenate([c - n + np.arange(1, n + 1) for n, c in zip(new, klen)])
        s.update(q=_normal(g, (T, H, dn + dr), dt), k=_normal(g, (S, H, dn), dt),
                 tail=_normal(g, (S, dr), dt) if dr else None,
                 v=_normal(g, (S, H, dv), dt, 0.5 * torch.randn(dv, generator=g, device=DEV)),
                 token_starts=_i32(np.concatenate([[0], np.cumsum(new)])),
                 key_starts=_i32(np.concatenate([[0], np.cumsum(klen)])), ends=_i32(ends),
                 longest=(int(new.max()), int(klen.max())), scale=1.25 / math.sqrt(dn + dr))
    else:
        W, T, H, dl = case["ranks"], case["tokens"], case["heads"], case["latent"]
        lse = torch.randn(W, T, H, generator=g, device=DEV) * 2 + 8
        lse[rng.randint(W), :, ::3] = -math.inf  # a rank that held none of the selected rows
        s.update(parts=_normal(g, (W, T, H, dl), dt), lse=lse)
    return s


# --- one pass ---------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_radix_gb300 as satk
    c = s["case"]
    op = c["op"]
    if op == "tables":
        t = satk.step_tables(s["context"], s["new"], s["free"], s["table"], tokens=s["tokens"],
                             block_size=c["block"], stride_rows=c["block"], W=c["ranks"],
                             dcp_rank=s["rank"], drafted=c["drafted"])
        return [s["table"], t.token_starts, t.lens, t.req_id, t.positions, t.row_ends, t.slots,
                t.blocks_used]
    if op == "store":
        return satk.latent_store(s["latent"], s["tail"], s["slots"], s["cache"],
                                 weight=s["weight"], eps=EPS,
                                 cos_sin=s["cos_sin"] if c["tail"] else None,
                                 positions=s["positions"] if c["tail"] else None,
                                 interleaved=c["interleaved"])
    if op == "attend":
        return satk.latent_attend(s["q"], s["cache"], s["req"], s["table"], s["ends"],
                                  block_size=c["block"], stride_rows=c["block"],
                                  latent_dim=c["latent"], scale=s["scale"], tree=s["tree"])
    if op == "rows":
        return satk.latent_attend_rows(s["q"], s["cache"], s["rows"], counts=s["counts"],
                                       latent_dim=c["latent"], scale=s["scale"])
    if op == "expanded":
        return satk.latent_attend_expanded(s["q"], s["k"], s["tail"], s["v"], s["token_starts"],
                                           s["key_starts"], s["ends"], scale=s["scale"])
    return satk.latent_merge(s["parts"], s["lse"])


def _local(p, W, rank):
    """How many of the first p tokens rank `rank` of W holds (token g: g % W)."""
    return torch.div(p + (W - 1 - rank), W, rounding_mode="floor")


def _attention(q, keys, values, visible, scale):
    """softmax(scale q keys^T) values over the visible keys, and the logarithm of
    the sum: q [G, M, D], keys [G, L, D], values [G, L, dv], visible [G, M, L]."""
    s = torch.matmul(q, keys.transpose(1, 2)) * scale
    s = torch.where(visible, s, -math.inf)
    m = s.amax(2, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(2, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total == 0, 1.0, total)
    return out, (m + torch.log(total)).squeeze(2)


def _run_plain(s):
    return globals()["_plain_" + s["case"]["op"]](s)


def _plain_tables(s):
    c = s["case"]
    W, B, rank, T = c["ranks"], c["block"], s["rank"], s["tokens"]
    ctx, new, table = s["context"].long(), s["new"].long(), s["table"]
    R, width = table.shape
    starts = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    have = _cdiv(_local(ctx, W, rank), B)
    lens = _local(ctx + new, W, rank)
    need = _cdiv(lens, B)
    base = (need - have).cumsum(0) - (need - have)
    col = torch.arange(width, device=DEV)[None]
    fresh = s["free"][(base[:, None] + col - have[:, None]).clamp(0, len(s["free"]) - 1)]
    table.copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), fresh, table))
    t = torch.arange(T, device=DEV)
    real = t < starts[-1]
    req = torch.where(real, torch.searchsorted(starts, t, right=True) - 1, 0)
    p = torch.where(real, ctx[req] + t - starts[req], 0)
    ends = _local(ctx[req], W, rank) if c["drafted"] else _local(p + 1, W, rank)
    ends = torch.where(real, ends, 0)
    l = torch.div(p, W, rounding_mode="floor")
    slot = table[req, (l // B).clamp(max=width - 1)].long() * B + l % B
    slot = torch.where(real & (p % W == rank), slot, -1)
    return [table, starts.int(), lens.int(), req.int(), p.int(), ends.int(), slot.int(),
            (need - have).sum().int().reshape(1)]


def _plain_store(s):
    c = s["case"]
    x, dr = s["latent"].float(), c["tail"]
    row = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"]
    if dr:
        y = s["tail"].float()
        cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, 1)
        a, b = (y[:, 0::2], y[:, 1::2]) if c["interleaved"] else y.chunk(2, 1)
        u, v = a * cos - b * sin, a * sin + b * cos
        rot = torch.stack([u, v], 2).flatten(1) if c["interleaved"] else torch.cat([u, v], 1)
        row = torch.cat([row, rot], 1)
    cache, slots = s["cache"], s["slots"].long()
    # a token that another rank holds writes again what the first kept one does
    kept = slots >= 0
    t = torch.where(kept, torch.arange(len(slots), device=DEV), kept.int().argmax())
    cache[slots[t]] = row.to(cache.dtype)[t]
    return cache


def _plain_attend(s):
    c = s["case"]
    R, n, H, dl, B = c["requests"], c["new"], c["heads"], c["latent"], c["block"]
    table, D = s["table"].long(), s["q"].shape[2]
    L = c["context"] + n
    j = torch.arange(L, device=DEV)
    keys = s["cache"][table[:, (j // B).clamp(max=table.shape[1] - 1)] * B + j % B].float()
    ends = s["ends"].long().view(R, n, 1)
    visible = j < ends
    if s["tree"] is not None:
        bit = (j - ends).clamp(0, 32 * s["tree"].shape[1] - 1)
        words = s["tree"].view(R, n, -1).long().gather(2, bit // 32)
        visible = visible | ((j >= ends) & (j - ends < 32 * s["tree"].shape[1])
                             & ((words >> (bit % 32)) & 1).bool())
    visible = visible[:, :, None].expand(R, n, H, L).reshape(R, n * H, L)
    out, lse = _attention(s["q"].float().view(R, n * H, D), keys, keys[..., :dl], visible,
                          s["scale"])
    return out.view(R * n, H, dl).to(s["q"].dtype), lse.view(R * n, H)


def _plain_rows(s):
    c = s["case"]
    rows = s["rows"].long()
    keys = s["cache"][rows.clamp(min=0)].float()
    k = rows.shape[1]
    visible = (rows >= 0) & (torch.arange(k, device=DEV) < s["counts"][:, None])
    out, lse = _attention(s["q"].float(), keys, keys[..., :c["latent"]],
                          visible[:, None].expand(-1, c["heads"], -1), s["scale"])
    return out.to(s["q"].dtype), lse


def _plain_expanded(s):
    (n, m), q, k, v = s["longest"], s["q"].float(), s["k"].float(), s["v"].float()
    if s["tail"] is not None:
        k = torch.cat([k, s["tail"].float()[:, None].expand(-1, k.shape[1], -1)], 2)
    ts, ks = s["token_starts"].long(), s["key_starts"].long()
    H, R = q.shape[1], len(ts) - 1
    i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    at = (ts[:-1, None] + i).clamp(max=q.shape[0] - 1)
    key_at = (ks[:-1, None] + j).clamp(max=k.shape[0] - 1)
    visible = (j < s["ends"].long()[at][..., None]) & (j < (ks[1:] - ks[:-1])[:, None, None])

    def heads_first(x, where):
        return x[where].transpose(1, 2).reshape(R * H, where.shape[1], -1)
    out, lse = _attention(heads_first(q, at), heads_first(k, key_at), heads_first(v, key_at),
                          visible.repeat_interleave(H, 0), s["scale"])
    t = torch.arange(q.shape[0], device=DEV)
    r = torch.searchsorted(ts, t, right=True) - 1
    out = out.view(R, H, n, -1).transpose(1, 2)[r, t - ts[r]]
    return out.to(s["q"].dtype), lse.view(R, H, n).transpose(1, 2)[r, t - ts[r]]


def _plain_merge(s):
    m = s["lse"].amax(0)
    w = torch.exp(s["lse"] - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(0)
    parts = torch.where(w[..., None] > 0, s["parts"].float() * w[..., None], 0.0)
    out = parts.sum(0) / torch.where(total == 0, 1.0, total)[..., None]
    return out.to(s["parts"].dtype), m + torch.log(total)


# --- the definition in 64 bits ---------------------------------------------

def _softmax_64(q, keys, values, scale):
    """One token group over exactly the keys it sees: q [M, D], keys [N, D]."""
    if keys.shape[0] == 0:
        return (torch.zeros(q.shape[0], values.shape[1], dtype=torch.float64, device=DEV),
                torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=DEV))
    s = (q @ keys.T) * scale
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ values, lse


def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return None
    s = prepare(case, seed)
    if op == "store":
        cache = s["cache"].double()
        dr = case["tail"]
        slots = s["slots"].cpu().numpy()
        x = s["latent"].double()
        norm = x / torch.sqrt((x ** 2).sum(1, keepdim=True) / case["latent"] + EPS)
        y = [norm * s["weight"].double()]
        if dr:
            tail = s["tail"].double()
            half = dr // 2
            one = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1)
            two = one + (1 if case["interleaved"] else half)
            z = torch.complex(tail[:, one], tail[:, two])
            cs = s["cos_sin"].double()[s["positions"].long()]
            z = z * torch.complex(cs[:, :half], cs[:, half:])
            rot = torch.empty_like(tail)
            rot[:, one], rot[:, two] = z.real.contiguous(), z.imag.contiguous()
            y.append(rot)
        keep = torch.from_numpy(np.nonzero(slots >= 0)[0]).to(DEV)
        cache[s["slots"].long()[keep]] = torch.cat(y, 1)[keep]
        return cache
    if op == "merge":
        lse = s["lse"].double()
        total = torch.logsumexp(lse, 0)
        return torch.einsum("wth,wthd->thd", torch.exp(lse - total), s["parts"].double()), total
    if op == "expanded":
        ts, ks = s["token_starts"].tolist(), s["key_starts"].tolist()
        T, H = s["q"].shape[:2]
        out = torch.zeros(T, H, case["value"], dtype=torch.float64, device=DEV)
        lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for r in range(len(ts) - 1):
            a, b, lo, hi = ts[r], ts[r + 1], ks[r], ks[r + 1]
            hide = torch.arange(hi - lo, device=DEV)[None] >= s["ends"][a:b].long()[:, None]
            for h in range(H):
                w = s["q"][a:b, h, :case["nope"]].double() @ s["k"][lo:hi, h].double().T
                if s["tail"] is not None:
                    w += s["q"][a:b, h, case["nope"]:].double() @ s["tail"][lo:hi].double().T
                w = (w * s["scale"]).masked_fill_(hide, -math.inf)
                lse[a:b, h] = torch.logsumexp(w, 1)
                out[a:b, h] = torch.exp(w - lse[a:b, h, None]) @ s["v"][lo:hi, h].double()
        return out, lse
    T, H = s["q"].shape[:2]
    dl = case["latent"]
    out = torch.zeros(T, H, dl, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    if op == "rows":
        rows, counts = s["rows"].cpu(), s["counts"].tolist()
    else:
        table, ends, B = s["table"].cpu().long(), s["ends"].tolist(), case["block"]
        words = s["tree"].cpu().numpy().view(np.uint32) if s["tree"] is not None else None
    for t in range(T):
        if op == "rows":
            at = rows[t, :counts[t]].long()
        else:
            j = list(range(ends[t]))
            if words is not None:
                j += [ends[t] + b for b in range(32 * words.shape[1])
                      if int(words[t, b // 32]) >> (b % 32) & 1]
            j = torch.tensor(j, dtype=torch.long)
            at = table[t // case["new"], j // B] * B + j % B
        keys = s["cache"][at.to(DEV)].double()
        out[t], lse[t] = _softmax_64(s["q"][t].double(), keys, keys[:, :dl], s["scale"])
    return out, lse
