"""Timed cases of the operators that train an indexer and the attention it
selects for: the distillation loss over a teacher's top entries with its
gradient, the attention's weights over selected cache rows (what an indexer is
distilled from), and the backward pass of the expanded prompt attention.

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
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --- cases ------------------------------------------------------------------

def listed():
    return [
        # a small batch against the top of a teacher's vocabulary: where latency counts
        dict(name="loss_small", op="loss", rows=16, cols=8192, k=64, kind="logits", scope="row",
             temperature=2.0, causal=False, dtype="bf16"),
        # an indexer's dense stage over a prompt chunk: causal rows of fp32 logits
        dict(name="loss_chunk", op="loss", rows=4096, cols=51200, k=512, kind="weights",
             scope="row", temperature=1.0, causal=True, dtype="fp32"),
        # an indexer's sparse stage: the softmax goes over the selected columns alone
        dict(name="loss_listed", op="loss", rows=4096, cols=25600, k=512, kind="weights",
             scope="listed", temperature=1.0, causal=True, dtype="bf16"),
        # the gradient of a model's logits against stored top entries of a teacher
        dict(name="grad_vocab", op="grad", rows=2048, cols=102400, k=64, kind="probs",
             scope="row", temperature=1.0, causal=False, dtype="bf16"),
        # a few long rows of odd length, many entries each
        dict(name="grad_few", op="grad", rows=4, cols=131071, k=2048, kind="logits", scope="row",
             temperature=1.5, causal=False, dtype="bf16"),
        # the sparse stage's gradient, zero outside the selected columns
        dict(name="grad_listed", op="grad", rows=4096, cols=8192, k=512, kind="weights",
             scope="listed", temperature=1.0, causal=True, dtype="fp32"),
        # one token's selected rows: the smallest call
        dict(name="weights_single", op="weights", tokens=1, context=8192, k=512, heads=20,
             latent=256, tail=64, dtype="bf16"),
        # tokens of one sequence over the rows that each selected of it
        dict(name="weights_batch", op="weights", tokens=512, context=16384, k=2048, heads=64,
             latent=512, tail=32, dtype="bf16"),
        # a few ragged prompts, none with a context, whose lse goes on into a join
        dict(name="expanded_prompts", op="expanded", requests=5, new=391, context=0, heads=12,
             nope=64, tail=32, value=64, dlse=True, dtype="fp16"),
        # longer prompts without a rotated tail
        dict(name="expanded_plain", op="expanded", requests=3, new=2900, context=0, heads=8,
             nope=128, tail=0, value=128, dlse=False, dtype="bf16"),
        # a prompt chunk of 4096 tokens whose keys are 8192 columns
        dict(name="expanded_chunk", op="expanded", requests=1, new=4096, context=4096, heads=16,
             nope=128, tail=64, value=128, dlse=False, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_one(rng):
    op = rng.choice(["loss", "grad", "weights", "expanded"])
    tail = rng.choice([0, 16, 32, 48, 64])
    if op in ("loss", "grad"):
        cols = _log_int(rng, 64, 131072)
        return dict(op=op, rows=_log_int(rng, 1, 4096), cols=cols,
                    k=min(_log_int(rng, 1, 2048), cols),
                    kind=rng.choice(["logits", "weights", "probs"]),
                    scope=rng.choice(["row", "listed"]), temperature=rng.choice([0.5, 1.0, 2.0]),
                    causal=rng.random() < 0.5, dtype=rng.choice(["fp32", "bf16", "fp16"]))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "weights":
        return dict(op=op, tokens=_log_int(rng, 1, 512), context=_log_int(rng, 64, 65536),
                    k=_log_int(rng, 16, 2048), heads=_log_int(rng, 1, 128),
                    latent=16 * _log_int(rng, 2, 32), tail=tail, dtype=dtype)
    return dict(op=op, requests=_log_int(rng, 1, 12), new=_log_int(rng, 1, 4096),
                context=rng.choice([0, _log_int(rng, 1, 4096)]), heads=_log_int(rng, 1, 32),
                nope=16 * rng.randint(2, 8), tail=tail, value=16 * rng.randint(2, 8),
                dlse=rng.random() < 0.3, dtype=dtype)


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

def _row_ends(case):
    """Visible columns of each row: all, or growing by one a row up to all."""
    n, cols = case["rows"], case["cols"]
    if not case["causal"]:
        return np.full(n, cols, dtype=np.int64)
    return np.maximum(1, cols - n + 1 + np.arange(n))


def _new_lens(case):
    """New tokens of each request: the case's `new` and below, one at least."""
    R, n = case["requests"], case["new"]
    return np.maximum(1, np.linspace(n, max(1, n // 3), R).astype(np.int64))


def _counts(case):
    """Selected rows of each token: k, or fewer for every fifth token and where
    the context is shorter than k."""
    n = min(case["k"], case["context"])
    return np.where(np.arange(case["tokens"]) % 5 == 4, n - n // 3, n)


def work(case):
    op = case["op"]
    if op in ("loss", "grad"):
        n, size = case["rows"], 4 if case["dtype"] == "fp32" else 2
        ends = _row_ends(case)
        entries = int(np.minimum(ends, case["k"]).sum())
        read = int(ends.sum()) if case["scope"] == "row" else entries
        flops = 4 * read + 8 * entries
        if op == "loss":
            return {"bytes": read * size + 8 * entries + 12 * n, "flops": flops}
        return {"bytes": (read + n * case["cols"]) * size + 8 * entries + 12 * n, "flops": flops}
    if op == "weights":
        H, D = case["heads"], case["latent"] + case["tail"]
        total = int(_counts(case).sum())
        io = case["tokens"] * H * (2 * D + 4) + 4 * case["tokens"] * (case["k"] + 1)
        return {"bytes": min(total, case["context"]) * D * 2 + io + 4 * total,
                "flops": 2 * total * H * D}
    H, D, dv = case["heads"], case["nope"] + case["tail"], case["value"]
    n, c = _new_lens(case), case["context"]
    T, S = int(n.sum()), int((n + c).sum())
    pairs = int((n * c + n * (n + 1) // 2).sum())
    keys = S * (H * (case["nope"] + dv) + case["tail"]) * 2
    return {"bytes": T * H * ((2 * D + 2 * dv) * 2 + 4 + 4 * case["dlse"]) + 2 * keys,
            "flops": 2 * pairs * H * (3 * D + 2 * dv)}


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


def prepare(case, seed):
    op = case["op"]
    rng = np.random.RandomState(seed % (1 << 32))
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if op in ("loss", "grad"):
        n, cols, k = case["rows"], case["cols"], case["k"]
        ends = _i32(_row_ends(case))
        logits = _normal(g, (n, cols), dt).mul_(2.5)
        # the teacher agrees with the student up to noise
        col = torch.arange(cols, device=DEV)
        teacher = logits + torch.empty_like(logits).normal_(generator=g)
        teacher = torch.where(col < ends[:, None], teacher, -math.inf)
        top = teacher.topk(k, dim=1)
        ids, order = torch.where(top.values > -math.inf, top.indices, cols).sort(dim=1)
        x = top.values.gather(1, order).float()
        if case["kind"] != "logits":
            # weights as attention sums them; probabilities with some mass elsewhere
            x = torch.exp(x - x.amax(1, keepdim=True))
            if case["kind"] == "probs":
                x = x / (1.25 * x.sum(1, keepdim=True))
        s.update(logits=logits, ends=ends if case["causal"] else None,
                 ids=torch.where(ids < cols, ids, -1).int().contiguous(), teacher=x.contiguous())
        if op == "grad":
            s.update(lse=_plain_loss(s)[1], dloss=torch.rand(n, generator=g, device=DEV) + 0.5)
    elif op == "weights":
        T, H, D, k = case["tokens"], case["heads"], case["latent"] + case["tail"], case["k"]
        L = case["context"]
        counts = _i32(_counts(case))
        pick = torch.rand(T, L, generator=g, device=DEV).topk(min(k, L), dim=1).indices
        rows = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        rows[:, :pick.shape[1]] = pick.int()
        rows[torch.arange(k, device=DEV)[None] >= counts[:, None]] = -1
        off = 0.5 * torch.randn(D, generator=g, device=DEV)
        s.update(q=_normal(g, (T, H, D), dt), cache=_normal(g, (L, D), dt, off), rows=rows,
                 counts=counts, scale=1.25 / math.sqrt(D))
        s["lse"] = _lse(_row_scores(s), 2)
    else:
        H, dn, dr, dv = case["heads"], case["nope"], case["tail"], case["value"]
        new = _new_lens(case)[rng.permutation(case["requests"])]
        klen = new + case["context"]
        T, S = int(new.sum()), int(klen.sum())
        ends = np.concatenate([c - n + np.arange(1, n + 1) for n, c in zip(new, klen)])
        s.update(q=_normal(g, (T, H, dn + dr), dt), k=_normal(g, (S, H, dn), dt),
                 tail=_normal(g, (S, dr), dt) if dr else None,
                 v=_normal(g, (S, H, dv), dt, 0.5 * torch.randn(dv, generator=g, device=DEV)),
                 dout=_normal(g, (T, H, dv), dt),
                 token_starts=_i32(np.concatenate([[0], np.cumsum(new)])),
                 key_starts=_i32(np.concatenate([[0], np.cumsum(klen)])), ends=_i32(ends),
                 longest=(int(new.max()), int(klen.max())), scale=1.25 / math.sqrt(dn + dr),
                 dlse=torch.randn(T, H, generator=g, device=DEV) if case["dlse"] else None)
        w = _where(s)
        scores, v = _scores(s, w), _heads_first(s["v"].float(), w["keys"])
        lse = _lse(scores, 2)
        out = torch.matmul(torch.exp(scores - lse[..., None]), v)
        s["out"], s["lse"] = _tokens_first(out, w).to(dt), _tokens_first(lse[..., None], w)[..., 0]
        s["lse"] = s["lse"].contiguous()
    return s


# --- one pass ---------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_attention_indexer_radix_gb300 as satk
    c = s["case"]
    if c["op"] in ("loss", "grad"):
        how = dict(kind=c["kind"], scope=c["scope"], temperature=c["temperature"],
                   row_ends=s["ends"])
        if c["op"] == "loss":
            return satk.distill_loss(s["logits"], s["ids"], s["teacher"], **how)
        return satk.distill_grad(s["logits"], s["ids"], s["teacher"], s["lse"], s["dloss"], **how)
    if c["op"] == "weights":
        return satk.latent_rows_weights(s["q"], s["cache"], s["rows"], s["lse"], scale=s["scale"],
                                        counts=s["counts"])
    return satk.latent_attend_expanded_grad(
        s["dout"], s["q"], s["k"], s["tail"], s["v"], s["out"], s["lse"], s["token_starts"],
        s["key_starts"], s["ends"], scale=s["scale"], dlse=s["dlse"])


def _run_plain(s):
    return globals()["_plain_" + s["case"]["op"]](s)


def _lse(x, dim):
    m = x.amax(dim, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    return (m + torch.log(torch.exp(x - m).sum(dim, keepdim=True))).squeeze(dim)


def _entries(s):
    """Columns of the entries, which of them count, and the teacher's share p."""
    c, x = s["case"], s["teacher"]
    cols = s["logits"].shape[1]
    ids = s["ids"].long()
    ends = s["ends"].long()[:, None] if s["ends"] is not None else cols
    live = (ids >= 0) & (ids < ends)
    if c["kind"] == "logits":
        x = torch.where(live, x / c["temperature"], -math.inf)
        m = x.amax(1, keepdim=True)
        x = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    else:
        x = torch.where(live, x.clamp(min=0), 0.0)
    if c["kind"] != "probs":
        total = x.sum(1, keepdim=True)
        x = x / torch.where(total == 0, 1.0, total)
    return ids.clamp(0, cols - 1), live, x


def _visible(s):
    """Scores over the temperature, -inf behind the rows' ends."""
    x = s["logits"].float() / s["case"]["temperature"]
    if s["ends"] is None:
        return x
    col = torch.arange(x.shape[1], device=DEV)
    return torch.where(col < s["ends"][:, None], x, -math.inf)


def _plain_loss(s):
    ids, live, p = _entries(s)
    picked = s["logits"].gather(1, ids).float() / s["case"]["temperature"]
    if s["case"]["scope"] == "row":
        lse = _lse(_visible(s), 1)
    else:
        lse = _lse(torch.where(live, picked, -math.inf), 1)
    log_p = torch.log(torch.where(p > 0, p, 1.0))
    loss = torch.where(p > 0, p * (log_p - picked + lse[:, None]), 0.0).sum(1)
    return loss, lse


def _plain_grad(s):
    ids, live, p = _entries(s)
    tau, lse = s["case"]["temperature"], s["lse"][:, None]
    g = (s["dloss"] / tau)[:, None]
    mass = p.sum(1, keepdim=True)
    if s["case"]["scope"] == "row":
        grad = torch.exp(_visible(s) - lse) * (g * mass)
        grad.scatter_add_(1, ids, -g * p)
    else:
        picked = s["logits"].gather(1, ids).float() / tau
        q = torch.where(live, torch.exp(picked - lse), 0.0)
        grad = torch.zeros(s["logits"].shape, device=DEV)
        grad.scatter_add_(1, ids, g * (mass * q - p))
    return grad.to(s["logits"].dtype)


def _row_scores(s):
    """Scores [T, H, k] of the selected rows, -inf where an entry is skipped."""
    rows = s["rows"].long()
    keys = s["cache"][rows.clamp(min=0)].float()
    live = (rows >= 0) & (torch.arange(rows.shape[1], device=DEV) < s["counts"][:, None])
    x = torch.matmul(s["q"].float(), keys.transpose(1, 2)) * s["scale"]
    return torch.where(live[:, None], x, -math.inf)


def _plain_weights(s):
    return torch.exp(_row_scores(s) - s["lse"][..., None]).mean(1)


def _where(s):
    """The tokens and keys of each request side by side, and what sees what."""
    n, m = s["longest"]
    ts, ks = s["token_starts"].long(), s["key_starts"].long()
    i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    tokens = ts[:-1, None] + i
    real = tokens < ts[1:, None]
    tokens = tokens.clamp(max=s["q"].shape[0] - 1)
    keys = ks[:-1, None] + j
    held = keys < ks[1:, None]
    keys = keys.clamp(max=s["k"].shape[0] - 1)
    seen = (j < s["ends"].long()[tokens][..., None]) & held[:, None] & real[..., None]
    return dict(tokens=tokens, real=real, keys=keys, held=held, seen=seen)


def _heads_first(x, where):
    """[N, H, w] as [R * H, longest, w]."""
    return x[where].transpose(1, 2).reshape(-1, where.shape[1], x.shape[2])


def _rows_back(x, real):
    """[R * H, longest, w] as [N, H, w], the requests' rows one after the other."""
    R, n = real.shape
    return x.view(R, -1, n, x.shape[2]).transpose(1, 2)[real]


def _tokens_first(x, w):
    return _rows_back(x, w["real"])


def _full_keys(s):
    k = s["k"].float()
    if s["tail"] is None:
        return k
    return torch.cat([k, s["tail"].float()[:, None].expand(-1, k.shape[1], -1)], 2)


def _scores(s, w):
    q, k = _heads_first(s["q"].float(), w["tokens"]), _heads_first(_full_keys(s), w["keys"])
    x = torch.matmul(q, k.transpose(1, 2)) * s["scale"]
    return torch.where(w["seen"].repeat_interleave(s["q"].shape[1], 0), x, -math.inf)


def _plain_expanded(s):
    w, dt = _where(s), s["q"].dtype
    tokens, keys = w["tokens"], w["keys"]
    lse = _heads_first(s["lse"][..., None], tokens)
    p = torch.exp(_scores(s, w) - lse)
    dout = _heads_first(s["dout"].float(), tokens)
    delta = (dout * _heads_first(s["out"].float(), tokens)).sum(2, keepdim=True)
    if s["dlse"] is not None:
        delta = delta - _heads_first(s["dlse"][..., None], tokens)
    dv = torch.matmul(p.transpose(1, 2), dout)
    dp = torch.matmul(dout, _heads_first(s["v"].float(), keys).transpose(1, 2))
    ds = p * (dp - delta) * s["scale"]
    dq = torch.matmul(ds, _heads_first(_full_keys(s), keys))
    dk = _rows_back(torch.matmul(ds.transpose(1, 2), _heads_first(s["q"].float(), tokens)),
                    w["held"])
    dn = s["k"].shape[2]
    dtail = dk[..., dn:].sum(1).to(dt) if s["tail"] is not None else None
    return (_tokens_first(dq, w).to(dt), dk[..., :dn].to(dt).contiguous(), dtail,
            _rows_back(dv, w["held"]).to(dt))


# --- the definition in 64 bits ---------------------------------------------

def _exact_rows(s, a, b):
    """Loss and normaliser, or the gradient, of the logits' rows [a, b)."""
    c = s["case"]
    tau, cols = c["temperature"], c["cols"]
    x, z = s["teacher"][a:b].double(), s["logits"][a:b].double() / tau
    ids = s["ids"][a:b].long()
    end = torch.full_like(ids[:, :1], cols) if s["ends"] is None else s["ends"][a:b, None].long()
    drop = (ids < 0) | (ids >= end)
    if c["kind"] == "logits":
        p = torch.softmax((x / tau).masked_fill(drop, -math.inf), 1)
    else:
        p = x.masked_fill(drop, 0.0)
        if c["kind"] == "weights":
            p = p / p.sum(1, keepdim=True)
    # the teacher's shares as a dense matrix, and how many entries a column has
    at = ids.masked_fill(drop, cols)
    share = torch.zeros(b - a, cols + 1, dtype=torch.float64, device=DEV)
    count = torch.zeros_like(share)
    share = share.scatter_add_(1, at, p)[:, :cols]
    count = count.scatter_add_(1, at, torch.ones_like(p))[:, :cols]
    if c["scope"] == "listed":
        log_q = z + torch.log(count)
    else:
        log_q = z.masked_fill(torch.arange(cols, device=DEV)[None] >= end, -math.inf)
    if c["op"] == "loss":
        lse = torch.logsumexp(log_q, 1)
        return (torch.special.xlogy(share, share) - share * (z - lse[:, None])).sum(1), lse
    q = torch.exp(log_q - s["lse"][a:b, None].double())
    return (s["dloss"][a:b, None].double() / tau * (share.sum(1, keepdim=True) * q - share),)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("loss", "grad"):
        n, step = case["rows"], max(1, (1 << 26) // case["cols"])  # blocks that fit the card
        parts = [_exact_rows(s, a, min(n, a + step)) for a in range(0, n, step)]
        whole = tuple(torch.cat(x) for x in zip(*parts))
        return whole if case["op"] == "loss" else whole[0]
    if case["op"] == "weights":
        out = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV)
        for t, n in enumerate(s["counts"].tolist()):
            keys = s["cache"][s["rows"][t, :n].long()].double()
            x = keys @ s["q"][t].double().T * s["scale"] - s["lse"][t].double()
            out[t, :n] = torch.exp(x).sum(1) / x.shape[1]
        return out
    dn, dr = case["nope"], case["tail"]
    ts, ks = s["token_starts"].tolist(), s["key_starts"].tolist()
    gq, gk, gt, gv = (None if x is None else torch.zeros(x.shape, dtype=torch.float64, device=DEV)
                      for x in (s["q"], s["k"], s["tail"], s["v"]))
    for r in range(len(ts) - 1):
        a, b, lo, hi = ts[r], ts[r + 1], ks[r], ks[r + 1]
        hide = torch.arange(hi - lo, device=DEV)[None] >= s["ends"][a:b].long()[:, None]
        for h in range(case["heads"]):
            q, do = s["q"][a:b, h].double(), s["dout"][a:b, h].double()
            key, val = s["k"][lo:hi, h].double(), s["v"][lo:hi, h].double()
            x = q[:, :dn] @ key.T
            if dr:
                x += q[:, dn:] @ s["tail"][lo:hi].double().T
            w = torch.exp(x.mul_(s["scale"]).sub_(s["lse"][a:b, h, None].double()))
            w.masked_fill_(hide, 0.0)
            gv[lo:hi, h] = w.T @ do
            row = torch.einsum("td,td->t", do, s["out"][a:b, h].double())
            if s["dlse"] is not None:
                row = row - s["dlse"][a:b, h].double()
            w *= (do @ val.T).sub_(row[:, None])
            w *= s["scale"]
            gk[lo:hi, h] = w.T @ q[:, :dn]
            gq[a:b, h, :dn] = w @ key
            if dr:
                gt[lo:hi] += w.T @ q[:, dn:]
                gq[a:b, h, dn:] = w @ s["tail"][lo:hi].double()
    return gq, gk, gt, gv
