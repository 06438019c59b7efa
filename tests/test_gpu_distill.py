"""distill_loss and distill_grad against their definitions in 64 bits.

Tolerances: an exponential's argument is a difference (or a product and a
normaliser) rounded a few times, so its value is off by (|argument| + 2) 2^-22 of
itself, exp2's own 2^-22 among that; sums of n terms in 32 bits add n / 512 + 20
roundings (a thread's share of a row, then a tree); a result's rounding to its type
is half a step.  Logarithms and the final sum round what they are given once."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from guards import guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0**-8, F16: 2.0**-11, F32: 2.0**-24}
LEAST = {BF16: 0.0, F16: 2.0**-25, F32: 0.0}  # half of the smallest step


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def definition(logits, ids, teacher, kind, scope, tau, ends, lse=None, dloss=None):
    """Loss, normaliser and (with dloss) gradient of one row after another in 64
    bits, with their tolerances."""
    rows, cols = logits.shape
    out = []
    for t in range(rows):
        end = cols if ends is None else min(max(int(ends[t]), 0), cols)
        e = ids[t].long()
        live = (e >= 0) & (e < end)
        e, x = e[live], teacher[t][live].double()
        z = logits[t].double() / tau
        if kind == "logits":
            d = (x - x.max()).abs() / tau if len(x) else x
            w = torch.exp((x - x.max()) / tau) if len(x) else x
            d = torch.where(w > 0, d, 0.0)
        else:
            w = x.clamp(min=0)
            d = torch.zeros_like(w)
        total = w.sum()
        p = w / total if kind != "probs" and total > 0 else w
        seen = z[:end] if scope == "row" else z[e]
        m = seen.max() if len(seen) else torch.tensor(-math.inf, dtype=torch.float64, device=DEV)
        n_lse = torch.logsumexp(seen, 0) if len(seen) else m
        q = torch.exp(seen - n_lse)
        far = torch.where(q > 0, q * (seen - m).abs(), 0.0).sum()
        log_l_tol = (2 + far) * 2.0**-21 + (cols / 512 + 20) * 2.0**-24
        lse_tol = log_l_tol + n_lse.abs() * 2.0**-22
        on = p > 0
        pe, ze, de = p[on], z[e][on], d[on]
        loss = (pe * (torch.log(pe) - ze + n_lse)).sum()
        size = torch.log(pe).abs() + (ze - m).abs() + (n_lse - m).abs() + 1
        loss_tol = (pe * size * (de + 2)).sum() * 2.0**-20 + pe.sum() * log_l_tol + 1e-30
        r = [loss, n_lse, loss_tol, lse_tol]
        if dloss is not None:
            g = float(dloss[t if dloss.numel() > 1 else 0]) / tau
            L = float(lse[t])
            grad = torch.zeros(cols, dtype=torch.float64, device=DEV)
            tol = torch.zeros_like(grad)
            if g != 0 and total > 0:
                at = torch.arange(end, device=DEV) if scope == "row" else e
                qv = torch.exp(z[at] - L) * p.sum()
                grad.index_add_(0, at, g * qv)
                tol.index_add_(0, at, abs(g) * qv * (z[at].abs() + abs(L) + 8) * 2.0**-21)
                grad.index_add_(0, e, -g * p)
                tol.index_add_(0, e, abs(g) * p * (d + 8) * 2.0**-20)
            u = U[logits.dtype]
            r += [grad, tol + u * grad.abs() + LEAST[logits.dtype]]
        out.append(r)
    return [torch.stack(x) for x in zip(*out)]


def close(got, want, tol, what):
    got = got.double()
    same = got == want
    off = torch.where(same, 0.0, (got - want).abs() - tol)
    assert not torch.isnan(off).any(), f"{what}: NaN"
    assert off.max().item() <= 0, f"{what}: beyond the tolerance by {off.max().item():.3g}"


def student(g, rows, cols, dtype, pad=0, offset=0, spread=2.5):
    ld = cols + pad
    buf = torch.empty(rows * ld + offset, dtype=dtype, device=DEV)
    buf.copy_(torch.randn(rows * ld + offset, generator=g, device=DEV) * spread)
    return buf[offset:].view(rows, ld)[:, :cols]


def entries(g, rows, cols, k, kind, ends=None, dtype=F32, holes=True):
    """Distinct random columns, some behind the rows' ends, some -1."""
    pick = torch.rand(rows, cols, generator=g, device=DEV).topk(min(k, cols), dim=1).indices.int()
    ids = torch.full((rows, k), -1, dtype=torch.int32, device=DEV)
    ids[:, :pick.shape[1]] = pick
    if holes and k > 3:
        ids[:, 2::7] = -1
    x = torch.randn(rows, k, generator=g, device=DEV) * 2
    if kind != "logits":
        x = torch.rand(rows, k, generator=g, device=DEV) / (k if kind == "probs" else 1)
    return ids, x.to(dtype)


def check(logits, ids, teacher, kind="logits", scope="row", tau=1.0, ends=None, dloss=None):
    how = dict(kind=kind, scope=scope, temperature=tau, row_ends=ends)
    rows, cols = logits.shape
    g = gen(9)
    if dloss is None:
        dloss = torch.rand(rows, generator=g, device=DEV) - 0.3
    loss_buf, loss_check = guarded((rows,), torch.int32)
    lse_buf, lse_check = guarded((rows,), torch.int32)
    loss, lse = satk.distill_loss(logits, ids, teacher, loss=loss_buf.view(F32),
                                  lse=lse_buf.view(F32), **how)
    grad = satk.distill_grad(logits, ids, teacher, lse, dloss, **how)
    want = definition(logits, ids, teacher, kind, scope, tau, ends, lse, dloss)
    close(lse, want[1], want[3], "lse")
    close(loss, want[0], want[2], "loss")
    close(grad, want[4], want[5], "gradient")
    loss_check("loss")
    lse_check("lse")
    return loss, lse, grad


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("kind", ["logits", "weights", "probs"])
@pytest.mark.parametrize("scope", ["row", "listed"])
def test_kinds_and_scopes(dtype, kind, scope):
    g = gen(1)
    for rows, cols, k, tau in ((7, 301, 20, 2.0), (3, 5000, 700, 0.5)):
        logits = student(g, rows, cols, dtype)
        ids, x = entries(g, rows, cols, k, kind)
        ends = torch.randint(1, cols + 1, (rows,), generator=g, device=DEV).int()
        check(logits, ids, x, kind, scope, tau)
        check(logits, ids, x, kind, scope, tau, ends)


@pytest.mark.parametrize("rows,cols,k", [
    (1, 1, 1), (1, 2, 4), (5, 3, 3), (2, 31, 31), (9, 257, 64), (1, 8191, 512), (1, 8192, 513),
    (2, 32768, 4096), (1, 32769, 100), (3, 65537, 2000), (1, 200003, 4096), (600, 77, 5),
    (1300, 4100, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sizes(rows, cols, k, dtype):
    g = gen(2)
    logits = student(g, rows, cols, dtype)
    ids, x = entries(g, rows, cols, k, "logits", holes=False)
    if rows > 10:
        loss, lse = satk.distill_loss(logits, ids, x)
        grad = satk.distill_grad(logits, ids, x, lse, torch.ones(1, device=DEV))
        for t in (0, 1, rows // 2, rows - 1):
            w = definition(logits[t:t + 1], ids[t:t + 1], x[t:t + 1], "logits", "row", 1.0, None,
                           lse[t:t + 1], torch.ones(1))
            close(lse[t:t + 1], w[1], w[3], "lse")
            close(loss[t:t + 1], w[0], w[2], "loss")
            close(grad[t:t + 1], w[4], w[5], "gradient")
        return
    check(logits, ids, x)
    check(logits, ids, x, scope="listed")


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (13, 2)])
def test_layouts(dtype, pad, offset):
    """Rows that start anywhere, of any stride; a gradient of another layout;
    what lies between the rows stays."""
    g = gen(3)
    logits = student(g, 6, 1003, dtype, pad, offset)
    ids, x = entries(g, 6, 1003, 50, "weights")
    wide = torch.zeros(6, 77, dtype=F32, device=DEV)
    wide[:, :50] = x
    _, lse, grad = check(logits, ids, x, "weights")
    for other in (0, 1, 4):
        n = 6 * (1003 + other) + 3
        buf = torch.full((n,), 7.0, dtype=dtype, device=DEV)
        out = buf[3:].view(6, 1003 + other)[:, :1003]
        got = satk.distill_grad(logits, ids, wide, lse, torch.ones(6, device=DEV), kind="weights",
                                k=50, out=out)
        again = satk.distill_grad(logits, ids, x, lse, torch.ones(1, device=DEV), kind="weights")
        assert got.data_ptr() == out.data_ptr() and torch.equal(out, again)
        assert (buf[:3] == 7).all()
        if other:
            assert (buf[3:].view(6, 1003 + other)[:, 1003:] == 7).all()


@pytest.mark.parametrize("teacher", [F32, BF16, F16])
def test_teacher_types(teacher):
    g = gen(4)
    logits = student(g, 5, 400, BF16)
    for kind in ("logits", "weights", "probs"):
        ids, x = entries(g, 5, 400, 40, kind, dtype=teacher)
        check(logits, ids, x, kind)


@pytest.mark.parametrize("dtype,cols", [(F32, 40000), (BF16, 1003), (F16, 70001)])
@pytest.mark.parametrize("scope", ["row", "listed"])
def test_gradient_in_place_of_the_scores(dtype, cols, scope):
    g = gen(5)
    logits = student(g, 4, cols, dtype, pad=5)
    ids, x = entries(g, 4, cols, 300, "logits")
    ids[:, 11] = ids[:, 10]
    ends = torch.tensor([cols, cols - 1, cols // 2, 0], dtype=torch.int32, device=DEV)
    _, lse, grad = check(logits, ids, x, scope=scope, ends=ends)
    dloss = torch.ones(4, device=DEV)
    want = satk.distill_grad(logits, ids, x, lse, dloss, scope=scope, row_ends=ends)
    got = satk.distill_grad(logits, ids, x, lse, dloss, scope=scope, row_ends=ends, out=logits)
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["logits", "weights", "probs"])
@pytest.mark.parametrize("scope", ["row", "listed"])
@pytest.mark.parametrize("k,distinct", [(16, 3), (600, 40), (4096, 1), (4096, 2048), (4096, 2500)])
def test_columns_named_more_than_once(kind, scope, k, distinct):
    g = gen(6)
    logits = student(g, 3, 5000, F32)
    ids = torch.randint(0, 5000, (3, distinct), generator=g, device=DEV).int()
    pick = torch.randint(0, distinct, (3, k), generator=g, device=DEV)
    ids = ids.gather(1, pick)
    _, x = entries(g, 3, 5000, k, kind)
    a = check(logits, ids, x, kind, scope)
    b = check(logits, ids, x, kind, scope)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_rows_without_entries_and_without_columns():
    g = gen(7)
    logits = student(g, 6, 100, BF16)
    ids, x = entries(g, 6, 100, 8, "logits")
    ids[1] = -1
    ids[2] = 99
    x[4] = -math.inf
    ends = torch.tensor([100, 100, 50, 0, 100, -3], dtype=torch.int32, device=DEV)
    logits[3] = math.nan  # nothing of it is visible
    logits[2, 50:] = math.inf
    dloss = torch.ones(6, device=DEV)
    for scope in ("row", "listed"):
        loss, lse = satk.distill_loss(logits, ids, x, row_ends=ends, scope=scope)
        grad = satk.distill_grad(logits, ids, x, lse, dloss, row_ends=ends, scope=scope)
        assert (loss[1:] == 0).all() and (grad[1:] == 0).all()
        assert torch.isneginf(lse[[3, 5]]).all() and torch.isfinite(loss[0])
        if scope == "row":
            assert torch.isfinite(lse[[1, 2, 4]]).all()
    # columns of no size, and no rows
    none = satk.distill_loss(logits[:, :0], ids, x)
    assert (none[0] == 0).all() and torch.isneginf(none[1]).all()
    assert satk.distill_grad(logits[:, :0], ids, x, none[1], dloss).shape == (6, 0)
    loss, lse = satk.distill_loss(logits[:0], ids[:0], x[:0])
    assert loss.shape == lse.shape == (0,)
    assert satk.distill_grad(logits[:0], ids[:0], x[:0], lse, loss).shape == (0, 100)


@pytest.mark.parametrize("scope", ["row", "listed"])
def test_values_that_are_not_finite(scope):
    g = gen(8)
    cols = 9000
    logits = student(g, 8, cols, F32)
    ids, x = entries(g, 8, cols, 30, "logits", holes=False)
    ids[:, 0] = torch.arange(8, device=DEV) + 10
    ends = torch.full((8,), cols - 5, dtype=torch.int32, device=DEV)
    logits[:, cols - 5:] = math.nan              # hidden from all
    logits[0, 10] = -math.inf                    # an entry that the student excludes
    logits[1, ids[1, 5].long() if scope == "listed" else 77] = math.nan
    logits[2, ids[2, 5].long() if scope == "listed" else 4000] = math.inf
    x[3, 4] = math.nan
    x[4, 4] = -math.inf                          # no share at all
    logits[5, (ids[5, 3].long() + 1) % 8000] = -math.inf
    ids[:, 29] = cols - 2                        # not visible
    loss, lse = satk.distill_loss(logits, ids, x, row_ends=ends, scope=scope)
    dloss = torch.ones(8, device=DEV)
    grad = satk.distill_grad(logits, ids, x, lse, dloss, row_ends=ends, scope=scope)
    assert torch.isposinf(loss[0]) and torch.isnan(loss[[1, 2, 3]]).all()
    assert torch.isfinite(loss[4:]).all() and torch.isfinite(lse[[0, 3, 4, 5, 6, 7]]).all()
    assert torch.isnan(lse[[1, 2]]).all()
    assert torch.isfinite(grad[[0, 4, 5, 6, 7]]).all()
    listed = ids[:, :29].long()
    assert torch.isnan(grad.gather(1, listed)[[1, 2, 3]]).all()
    assert (grad[:, cols - 5:] == 0).all()
    w = definition(logits[4:], ids[4:], x[4:], "logits", scope, 1.0, ends[4:], lse[4:], dloss[4:])
    close(loss[4:], w[0], w[2], "loss")
    close(grad[4:], w[4], w[5], "gradient")
    # rows whose loss nobody wants get zeros, whatever they hold
    dloss[:4] = 0
    grad = satk.distill_grad(logits, ids, x, lse, dloss, row_ends=ends, scope=scope)
    assert (grad[:4] == 0).all()


@pytest.mark.parametrize("scale", [1e-30, 1e4, 1e30])
def test_scores_of_any_size(scale):
    """Loss and lse keep their digits at any size; the gradient's shares are within
    [0, 1] and right where lse has digits behind the point."""
    g = gen(10)
    logits = student(g, 4, 3001, F32) * scale
    ids, x = entries(g, 4, 3001, 40, "weights")
    loss, lse = satk.distill_loss(logits, ids, x, kind="weights")
    w = definition(logits, ids, x, "weights", "row", 1.0, None)
    close(lse, w[1], w[3], "lse")
    close(loss, w[0], w[2], "loss")
    grad = satk.distill_grad(logits, ids, x, lse, torch.ones(1, device=DEV), kind="weights")
    assert torch.isfinite(grad).all() and grad.abs().max() <= 1.0 + 1e-5
    # a large offset shared by a row changes nothing but lse
    base = student(g, 4, 3001, F32).mul_(64).round_().div_(64)
    a = satk.distill_loss(base, ids, x, kind="weights")
    b = satk.distill_loss(base + 4096, ids, x, kind="weights")
    assert torch.equal(a[0], b[0])


def test_offsets_beyond_32_bits():
    ld = (1 << 30) + 8
    buf = torch.zeros(2 * ld + 4096, dtype=BF16, device=DEV)
    out = torch.zeros(2 * ld + 4096, dtype=BF16, device=DEV)
    g = gen(11)
    logits = buf.as_strided((3, 1000), (ld, 1))
    grad = out.as_strided((3, 1000), (ld, 1))
    logits.copy_(torch.randn(3, 1000, generator=g, device=DEV))
    ids, x = entries(g, 3, 1000, 20, "logits")
    loss, lse = satk.distill_loss(logits, ids, x)
    satk.distill_grad(logits, ids, x, lse, torch.ones(3, device=DEV), out=grad)
    w = definition(logits, ids, x, "logits", "row", 1.0, None, lse, torch.ones(3))
    close(loss, w[0], w[2], "loss")
    close(grad, w[4], w[5], "gradient")


def test_gradient_against_differences():
    """The gradient along a direction against differences of the loss in 64 bits."""
    g = gen(12)
    for kind in ("logits", "weights", "probs"):
        for scope in ("row", "listed"):
            logits = student(g, 4, 700, F32)
            ids, x = entries(g, 4, 700, 60, kind)
            lse = satk.distill_loss(logits, ids, x, kind=kind, scope=scope, temperature=1.5)[1]
            grad = satk.distill_grad(logits, ids, x, lse, torch.ones(4, device=DEV), kind=kind,
                                     scope=scope, temperature=1.5)
            way = torch.randn(4, 700, generator=g, device=DEV).double()
            h = 1e-4

            def at(s):
                d = definition(logits.double() + s * way, ids, x, kind, scope, 1.5, None)
                return d[0]
            slope = (at(h) - at(-h)) / (2 * h)
            got = (grad.double() * way).sum(1)
            # h^2 of the third derivative, and the gradient's own 32 bits
            assert ((got - slope).abs() <= 1e-6 + 1e-5 * grad.abs().double().sum(1)).all()


def test_streams_graphs_and_two_calls_at_once():
    g = gen(13)
    logits = student(g, 8, 20000, BF16)
    ids, x = entries(g, 8, 20000, 256, "weights")
    dloss = torch.rand(8, generator=g, device=DEV)
    want = check(logits, ids, x, "weights", dloss=dloss)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            loss, lse = satk.distill_loss(logits, ids, x, kind="weights")
            got.append((loss, lse, satk.distill_grad(logits, ids, x, lse, dloss, kind="weights")))
    torch.cuda.synchronize()
    for r in got:
        for u, v in zip(r, want):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    loss, lse = torch.empty(8, device=DEV), torch.empty(8, device=DEV)
    out = torch.empty_like(logits)
    with torch.cuda.graph(graph):
        satk.distill_loss(logits, ids, x, kind="weights", loss=loss, lse=lse)
        satk.distill_grad(logits, ids, x, lse, dloss, kind="weights", out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[2]) and torch.equal(loss, want[0])


def test_one_value_of_dloss_for_every_row():
    g = gen(14)
    logits = student(g, 5, 333, F32)
    ids, x = entries(g, 5, 333, 10, "logits")
    lse = satk.distill_loss(logits, ids, x)[1]
    a = satk.distill_grad(logits, ids, x, lse, torch.full((5,), 0.25, device=DEV))
    for d in (torch.full((1,), 0.25, device=DEV), torch.tensor(0.25, device=DEV),
              torch.tensor(0.25, device=DEV).expand(5)):
        assert torch.equal(a, satk.distill_grad(logits, ids, x, lse, d))


def test_entries_as_the_selection_writes_them():
    """topk_rows' ids of the teacher's scores, its two ascending runs and -1 tails."""
    g = gen(15)
    teacher = student(g, 6, 600, F32).mul_(4).round_()
    ends = torch.tensor([600, 599, 64, 20, 3, 0], dtype=torch.int32, device=DEV)
    ids = satk.topk_rows(teacher, 64, row_ends=ends)
    x = teacher.gather(1, ids.long().clamp(min=0))
    check(student(g, 6, 600, BF16), ids, x, "logits", "row", 2.0, ends)
    check(student(g, 6, 600, BF16), ids, x, "logits", "listed", 2.0, ends)


def test_refusals():
    logits, ids = torch.zeros(4, 50, device=DEV), torch.zeros(4, 8, dtype=torch.int32, device=DEV)
    x, r = torch.zeros(4, 8, device=DEV), torch.zeros(4, device=DEV)
    bad = [
        dict(logits=logits.double()), dict(logits=logits.t()), dict(logits=logits[0]),
        dict(ids=ids.long()), dict(ids=ids[:3]), dict(x=x.double()), dict(x=x[:, :7]),
        dict(kind="mass"), dict(scope="all"), dict(temperature=0.0), dict(temperature=-1.0),
        dict(temperature=math.nan), dict(temperature=math.inf), dict(temperature=1e-45), dict(k=9),
        dict(k=0), dict(row_ends=ids[:, 0]), dict(row_ends=ids[:3, 0].contiguous()),
        dict(row_ends=r), dict(ids=torch.zeros(4, 4097, dtype=torch.int32, device=DEV),
                               x=torch.zeros(4, 4097, device=DEV))]
    for kw in bad:
        kw = dict(kw)
        args = [kw.pop("logits", logits), kw.pop("ids", ids), kw.pop("x", x)]
        with pytest.raises(satk.SatkError):
            satk.distill_loss(*args, **kw)
        with pytest.raises(satk.SatkError):
            satk.distill_grad(*args, r, r, **kw)
    for kw in (dict(loss=r[:3]), dict(lse=r.double())):
        with pytest.raises(satk.SatkError):
            satk.distill_loss(logits, ids, x, **kw)
    for lse, dloss, out in ((r[:3], r, None), (r, r[:2], None), (r, r.double(), None),
                            (r, torch.zeros(8, device=DEV)[::2], None), (r, r, logits[:, :49]),
                            (r, r, logits.bfloat16())):
        with pytest.raises(satk.SatkError):
            satk.distill_grad(logits, ids, x, lse, dloss, out=out)


def test_int_row_ends_from_numpy_and_default_k():
    ends = torch.from_numpy(np.array([5, 9], dtype=np.int32)).to(DEV)
    g = gen(16)
    logits = student(g, 2, 9, F16)
    ids = torch.tensor([[0, 4, 8], [8, 2, -1]], dtype=torch.int32, device=DEV)
    check(logits, ids, torch.rand(2, 3, generator=g, device=DEV), "probs", "row", 1.0, ends)
