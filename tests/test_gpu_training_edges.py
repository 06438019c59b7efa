"""Corners of the training calls: gradients of other layouts than the inputs', rows of
no size in clusters, lists of very small and very large weights, values and heads
that do not count, normalisers far from 0, short requests beside long ones.

Tolerances that are not those of the operators' own tests stand at each test."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from sparse_attention_indexer_radix_gb300 import build as satk_build
from test_gpu_distill import F32, check, entries, student
from test_gpu_distill import close as close_rows
from test_gpu_distill import definition as distilled
from test_gpu_expanded_grad import Case, close, definition
from test_gpu_latent import BF16, DEV, F16, U, gen, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    satk_build.build()


def placed(x, how):
    """A tensor like x, full of 7, that starts at an odd element or whose rows or
    heads lie an odd number of elements apart, and all of its memory."""
    base, heads, rows = {"base": (1, 0, 0), "heads": (0, 3, 0), "rows": (0, 0, 5)}[how]
    n, H, w = x.shape if x.dim() == 3 else (x.shape[0], 1, x.shape[1])
    ld_h = w + heads
    ld = H * ld_h + rows
    wide = torch.full((n * ld + 16,), 7.0, dtype=x.dtype, device=DEV)
    strides = (ld, ld_h, 1) if x.dim() == 3 else (ld, 1)
    return wide.as_strided(x.shape, strides, base), wide


@pytest.mark.parametrize("how", ["base", "heads", "rows"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", [
    (2, 128, 64, 128, [300, 77], [100, 0]), (3, 96, 48, 80, [129, 64, 250], [31, 0, 0]),
    (2, 192, 64, 128, [200, 33], [100, 0]), (1, 64, 0, 64, [400], [0]), (4, 16, 16, 16, [130], [5]),
    (2, 128, 64, 128, [2, 3, 8], [0, 400, 1100]), (2, 144, 64, 112, [8] * 9, [130] * 9)])
def test_gradients_of_another_layout_than_the_inputs(dtype, how, shape):
    """Aligned inputs, gradients that are not: the bits of aligned ones, whole, and
    nothing between their rows."""
    c = Case(gen(1), dtype, *shape, dlse=True)
    c.forward()
    want = c.grad()
    close(want, definition(c), "aligned")
    names = [n for n, x in zip(("dq", "dk", "dtail", "dv"), want) if x is not None]
    for _ in range(3):
        into = {n: placed(x, how) for n, x in zip(("dq", "dk", "dtail", "dv"), want) if n in names}
        got = c.grad(**{n: x for n, (x, _) in into.items()})
        for name, x, y in zip(("dq", "dk", "dtail", "dv"), got, want):
            assert x is y is None or torch.equal(x, y), name
        for name, (x, wide) in into.items():
            x.fill_(7.0)
            assert (wide == 7).all(), name


@pytest.mark.parametrize("scope", ["row", "listed"])
@pytest.mark.parametrize("rows", [1, 2, 7])
def test_wide_rows_with_little_to_see(rows, scope):
    """Rows shared by a cluster of which most CTAs have no column."""
    g = gen(2)
    cols = 131072
    logits = student(g, rows, cols, BF16)
    ids = torch.arange(16, device=DEV, dtype=torch.int32).repeat(rows, 1)
    x = torch.rand(rows, 16, generator=g, device=DEV)
    for ends in ([0] * rows, [1] * rows, [(5, 0, 4097, 1, 131072, 16, 131071)[i] for i in range(rows)]):
        ends = i32(ends)
        want = check(logits, ids, x, "weights", scope, 1.0, ends)
        for _ in range(20):
            got = satk.distill_loss(logits, ids, x, kind="weights", scope=scope, row_ends=ends)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_of_almost_2_31_columns():
    """Scores and a gradient of different alignment over the widest row there can be:
    every column is written once, nothing behind them."""
    cols = 2**31 - 1
    logits = torch.zeros(1, cols, dtype=BF16, device=DEV)
    wide = torch.full((cols + 16,), 7.0, dtype=BF16, device=DEV)
    out = wide[1:cols + 1].view(1, cols)
    ids, x = i32([[5, cols - 1, -1]]), torch.tensor([[1.0, 3.0, 9.0]], device=DEV)
    loss, lse = satk.distill_loss(logits, ids, x, kind="weights")
    want = math.log(cols)
    assert abs(lse.item() - want) <= 1e-5
    assert abs(loss.item() - (want + 0.25 * math.log(0.25) + 0.75 * math.log(0.75))) <= 1e-4
    dloss = torch.full((1,), float(cols), device=DEV)
    satk.distill_grad(logits, ids, x, lse, dloss, kind="weights", out=out)
    assert wide[0] == 7 and (wide[cols + 1:] == 7).all()
    for v, p in ((5, 0.25), (cols - 1, 0.75)):
        assert abs(out[0, v].item() / (1 - p * cols) - 1) <= 2.0**-7
        out[0, v] = 1.0
    for part in out[0].split(1 << 28):  # (shares of 1, within |lse| 2^-22 of themselves)
        assert (part == 1).all()


@pytest.mark.parametrize("shape", [(2, 128, 64, 128, [300, 77], [100, 0]), (3, 96, 48, 80, [129, 5], [31, 70]),
                                   (2, 128, 64, 128, [2, 3, 8], [0, 400, 1100])])
@pytest.mark.parametrize("how", ["base", None])
def test_a_given_up_wait_makes_gradients_nan(shape, how):
    """No wait is made to run out: the debug build, asked to, ends every CTA as after
    one.  Whole gradient rows are NaN, rows that nothing sees or no request has 0, and
    nothing between the rows is written; once nothing is asked for all is right again."""
    dbg = binding.load(satk_build.build(debug=True))
    c = Case(gen(10), BF16, *shape, spare=(20, 30))
    hidden = int(c.ks[1])  # the first request's last key
    c.ends[:int(c.ts[1])] = torch.clamp(c.ends[:int(c.ts[1])], max=hidden - 1)
    c.forward()
    names, into = ("dq", "dk", "dtail", "dv"), {}
    with binding.routed_to(dbg):
        dbg.satk_debug_flags(1)
        good = c.grad()
        if how:
            into = {n: placed(x, how) for n, x in zip(names, good)}
        dbg.satk_debug_flags(2)
        try:
            bad = c.grad(**{n: x for n, (x, _) in into.items()})
            torch.cuda.synchronize()
        finally:
            assert dbg.satk_debug_flags(1) == 256
        again = c.grad()
    close(good, definition(c), "good")
    T, S = int(c.ts[-1]), int(c.ks[-1])
    for name, x, end in zip(names, bad, (T, S, S, S)):
        assert torch.isnan(x[:end]).all() and (x[end:] == 0).all(), name
    for name, (x, wide) in into.items():
        x.fill_(7.0)
        assert (wide == 7).all(), name
    for x, y in zip(good, again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("size", [1e-44, 1e-39, 1e-30, 1e30, 3e38])
@pytest.mark.parametrize("scope", ["row", "listed"])
@pytest.mark.parametrize("k", [2, 600, 2100])
def test_weights_of_any_size(size, scope, k):
    """Shares of a sum that 32 bits hold badly, or not at all (the weights
    themselves are exact): those of their ratios."""
    g = gen(3)
    logits = student(g, 4, 5000, F32)
    ids, x = entries(g, 4, 5000, k, "weights", holes=False)
    x = x.double() * size
    x[0, 0], x[0, 1] = 1e-40, 3e-40
    x[1] *= torch.logspace(-20, 0, k, dtype=torch.float64, device=DEV)
    x[2, 1] = -1.0
    x[3, 0] = 1e-42
    ids[3, -1] = ids[3, 0]
    check(logits, ids, x.float(), "weights", scope)


def test_weights_of_any_size_in_16_bits():
    g = gen(4)
    logits = student(g, 3, 700, BF16)
    ids, x = entries(g, 3, 700, 40, "weights")
    for dtype, size in ((BF16, 1e-39), (BF16, 3e38), (F16, 1e-6), (F16, 60000.0)):
        check(logits, ids, (x * size).to(dtype), "weights")


@pytest.mark.parametrize("scope", ["row", "listed"])
@pytest.mark.parametrize("kind", ["logits", "weights", "probs"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_teacher_values_that_are_not_finite(kind, scope, value):
    """One among a row's entries makes its loss, and the gradient of its entries, NaN;
    one that does not count, and other rows, see nothing of it."""
    g = gen(5)
    for cols, k, again in ((900, 30, False), (3000, 700, True)):
        logits = student(g, 5, cols, F32)
        ids, x = entries(g, 5, cols, k, kind, holes=False)
        if again:
            ids[:, 7] = ids[:, 8]  # a column named twice
        ids[:, 3] = -1
        one = torch.ones(1, device=DEV)
        how = dict(kind=kind, scope=scope)
        clean = satk.distill_loss(logits, ids, x, **how)
        grad = satk.distill_grad(logits, ids, x, clean[1], one, **how)
        x[1, 8] = value
        x[2, 3] = value
        loss, lse = satk.distill_loss(logits, ids, x, **how)
        got = satk.distill_grad(logits, ids, x, lse, one, **how)
        assert torch.isnan(loss[1]) and torch.equal(lse, clean[1])
        assert torch.isnan(got[1][ids[1][ids[1] >= 0].long()]).all()
        keep = [0, 2, 3, 4]
        assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(got[keep], grad[keep])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,D", [(5, 96), (16, 64), (17, 544), (130, 192), (5, 35), (33, 17)])
def test_heads_that_saw_nothing_add_nothing(dtype, H, D):
    """A head whose lse is -inf adds 0 whatever its queries and the rows hold, and
    what fills a tile's heads up adds nothing to rows that are not finite: those have
    the weights that their scores, infinities too, have."""
    g = gen(6)
    q = torch.randn(3, H, D, generator=g, device=DEV).to(dtype)
    q = torch.where(q == 0, 1.0, q)
    cache = torch.randn(300, D, generator=g, device=DEV).to(dtype)
    rows = torch.randint(-1, 300, (3, 140), generator=g, device=DEV).int()
    rows = torch.where((rows == 7) | (rows == 9), 8, rows)
    lse = torch.randn(3, H, generator=g, device=DEV) + 4
    lse[0, 1:3] = -math.inf
    lse[2] = -math.inf
    call = lambda: satk.latent_rows_weights(q, cache, rows, lse, scale=0.2)  # noqa: E731
    clean = call()
    # queries of heads that saw nothing
    keep = q.clone()
    q[0, 1, 0], q[0, 2, 3] = math.nan, math.inf
    q[2, :, 1] = math.nan
    assert torch.equal(call(), clean) and (clean[2] == 0).all()
    q = keep
    # rows with one infinity: a weight of 1 or 0 a head
    cache[7, 2], cache[9, 4] = math.inf, -math.inf
    rows[:, 50], rows[:, 139] = 7, 9
    got = call()
    live = ~torch.isneginf(lse)
    for at, col, sign in ((50, 2, 1), (139, 4, -1)):
        want = (live & (q[:, :, col].float() * sign > 0)).double().sum(1) / H
        assert ((got[:, at].double() - want).abs() <= want * 2.0**-22).all()
    others = [j for j in range(140) if j not in (50, 139)]
    assert torch.equal(got[:, others], clean[:, others])
    # rows with a NaN: of every head that saw something
    cache[7, 2] = math.nan
    got = call()
    assert torch.isnan(got[:2, 50]).all() and got[2, 50] == 0
    assert torch.equal(got[:, others], clean[:, others])


@pytest.mark.parametrize("offset", [0.0, 300.0, -5000.0])
@pytest.mark.parametrize("scope", ["row", "listed"])
@pytest.mark.parametrize("tau", [1.0, 0.25, 0.7])
def test_shares_of_far_scores(offset, scope, tau):
    """The student's share is off by the roundings of s / tau - lse alone, not of a
    product with lse: 2^-24 of the difference d and, with a 1 / tau that is rounded,
    of s / tau; d log2(e) 3 more of |d| 2^-24, exp2 2^-22 (and 2^-24 for its use), the
    products with the row's factors and the sum with p 4 2^-24 of what they take."""
    g = gen(7)
    logits = student(g, 4, 3001, F32) + offset
    ids, x = entries(g, 4, 3001, 40, "weights", holes=False)
    how = dict(kind="weights", scope=scope, temperature=tau)
    _, lse = satk.distill_loss(logits, ids, x, **how)
    one = torch.ones(1, device=DEV)
    got = satk.distill_grad(logits, ids, x, lse, one, **how).double()
    at = ids.long()
    z = logits.double() / tau
    d = z - lse.double()[:, None]
    q = torch.exp(torch.clamp(d, max=0.0))
    p = (x.double() / x.double().sum(1, keepdim=True))
    listed = torch.zeros_like(q).scatter_(1, at, 1.0)
    if scope == "listed":
        q = q * listed
    share = torch.zeros_like(q).scatter_add_(1, at, p)
    inexact = 0.0 if tau in (1.0, 0.25) else 1.0
    tol = q * (d.abs() * 4 + z.abs() * inexact + 4 + 1 + 4) + share * (40 + 8)
    off = (got - (q - share) / tau).abs() - tol * 2.0**-24 / tau
    assert off.max().item() <= 1e-30


@pytest.mark.parametrize("H,D", [(16, 64), (64, 128), (150, 64), (3, 17)])
@pytest.mark.parametrize("offset", [0, 400, -3000])
def test_weights_of_far_scores(H, D, offset):
    """Products that are exact in 32 bits, so that only scale s - lse (2^-24 of the
    difference d), its product with log2(e) (3 |d| 2^-24), exp2 (2^-22 and 2^-24) and the
    sum over the heads (H + 2 roundings) are not."""
    g = gen(9)
    q = torch.randint(-4, 5, (3, H, D), generator=g, device=DEV).to(BF16)
    cache = torch.randint(-4, 5, (200, D), generator=g, device=DEV).to(BF16)
    q[..., 0], cache[:, 0] = 8.0, offset / 2.0  # (a share of the scores that all have)
    rows = torch.randint(0, 200, (3, 130), generator=g, device=DEV).int()
    keys = cache[rows.long()].double()
    x = torch.einsum("thd,tkd->thk", q.double(), keys) * 0.25
    lse = torch.logsumexp(x, 2).float()
    got = satk.latent_rows_weights(q, cache, rows, lse, scale=0.25).double()
    d = torch.clamp(x - lse.double()[..., None], max=0.0)
    w = torch.exp(d)
    tol = (w * (d.abs() * 4 + 5 + H + 2)).mean(1) * 2.0**-24
    assert ((got - w.mean(1)).abs() <= tol + 1e-37).all()


SHORT = [1, 5, 8, 16, 33, 64]


def beside(long, more=0, dtype=BF16):
    """Short requests, then `long` tokens in a request of their own and `more`
    requests of none; inputs that depend on the request alone."""
    new = SHORT + ([long] if long else []) + [0] * more
    context = [0, 3, 400, 1100, 64, 0] + ([40] if long else []) + [0] * more
    parts = [Case(gen(50 + r), dtype, 2, 64, 32, 64, [n], [c], dlse=True)
             for r, (n, c) in enumerate(zip(new, context)) if n]
    whole = Case(gen(50), dtype, 2, 64, 32, 64, new, context, dlse=True)
    for name in ("q", "k", "v", "tail", "dout", "dlse"):
        setattr(whole, name, torch.cat([getattr(p, name) for p in parts]))
    return whole, parts


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("long,more", [(1, 0), (65, 0), (700, 0), (4000, 0), (700, 300)])
def test_a_request_does_not_depend_on_the_others(dtype, long, more):
    """The bits of short requests, whatever else is in the call, and their exactness:
    P and dS as two operands each."""
    c, parts = beside(long, more, dtype)
    c.forward()
    got = c.grad()
    for r, p in enumerate(parts):
        p.forward()
        want = p.grad()
        if r < len(SHORT):
            close(want, definition(p, roundings=2), f"request {r} alone")
        t, s = slice(c.ts[r], c.ts[r + 1]), slice(c.ks[r], c.ks[r + 1])
        for x, y, at in zip(got, want, (t, s, s, s)):
            assert torch.equal(x[at], y), r
    if long <= 700:
        close(got, definition(c), "together")


@pytest.mark.parametrize("new,context", [([700], [60]), ([65], [0]), ([64], [200]), ([3], [9])])
def test_requests_of_no_tokens_change_nothing(new, context):
    c = Case(gen(8), BF16, 2, 128, 64, 128, new, context)
    c.forward()
    want = c.grad()
    for before, after in ((0, 255), (100, 0), (3, 40)):
        c.ts = np.concatenate([[0] * before, [0, new[0]], [new[0]] * after])
        n = new[0] + context[0]
        c.ks = np.concatenate([[0] * before, [0, n], [n] * after])
        for x, y in zip(c.grad(), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("H", [16, 128])
def test_a_cache_of_more_rows_than_an_entry_can_name(H):
    """Copies and gathers; the call is told of 2^33 rows, of which it is given the first."""
    g = gen(11)
    D = 576
    cache = torch.randn(200, D, generator=g, device=DEV).to(BF16)
    q = torch.randn(2, H, D, generator=g, device=DEV).to(BF16)
    rows = torch.randint(-1, 200, (2, 130), generator=g, device=DEV).int()
    lse = torch.full((2, H), 8.0, device=DEV)
    want = satk.latent_rows_weights(q, cache, rows, lse, scale=0.05)
    out = torch.full_like(want, math.nan)
    rc = binding.lib().satk_latent_rows_weights(
        q.data_ptr(), binding.SATK_BF16, 2, H, D, H * D, D, cache.data_ptr(), 2**33, D,
        rows.data_ptr(), 130, 130, None, 0.05, lse.data_ptr(), out.data_ptr(), 130, None,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(out, want)
