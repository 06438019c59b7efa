"""latent_rows_weights against its definition in 64 bits.

Tolerances: a score is off by ds (fp32 sums of D products: D 2^-23 scale sum
|q||k|), an exponent by (|score| + |lse| + 2) 2^-22 more, exp2 among it; H weights
are summed in 32 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from guards import guarded
from test_gpu_latent import BF16, DEV, F16, gen, i32, latent_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


def definition(q, cache, rows, counts, lse, scale):
    T, H, D = q.shape
    k = rows.shape[1]
    out = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(out)
    for t in range(T):
        n = k if counts is None else min(max(int(counts[t]), 0), k)
        live = torch.zeros(k, dtype=torch.bool, device=DEV)
        live[:n] = True
        live &= (rows[t] >= 0) & (rows[t] < cache.shape[0])
        if not live.any():
            continue
        keys = cache[rows[t][live].long()][:, :D].double()
        x, L = keys @ q[t].double().T * scale, lse[t].double()
        ds = (keys.abs() @ q[t].double().abs().T) * abs(scale) * D * 2.0**-23
        w = torch.where(torch.isneginf(L), 0.0, torch.exp(torch.clamp(x - L, max=0.0)))
        out[t, live] = w.mean(1)
        e = torch.where(w > 0, ds + (x.abs() + L.abs() + 2) * 2.0**-21 + H * 2.0**-24, 0.0)
        tol[t, live] = (w * e).mean(1) + 1e-38
    return out, tol


def close(got, want, tol, what=""):
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(off).any(), f"{what}: NaN"
    assert off.max().item() <= 0, f"{what}: beyond the tolerance by {off.max().item():.3g}"


def case(g, T, H, D, k, n_rows, dtype, ld=None, offset=0, counts=True):
    cache = latent_rows(g, n_rows, D, dtype, ld=ld, offset=offset)
    q = torch.randn(T, H, D, generator=g, device=DEV).to(dtype)
    rows = torch.randint(-1, n_rows, (T, k), generator=g, device=DEV).int()
    n = torch.randint(0, k + 1, (T,), generator=g, device=DEV).int() if counts else None
    return q, cache, rows, n


def run(q, cache, rows, counts, dl, scale, check_guard=True):
    _, lse = satk.latent_attend_rows(q, cache, rows, counts=counts, latent_dim=dl, scale=scale)
    T, k = rows.shape
    buf, guard = guarded((T, k), torch.int32)
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=scale, counts=counts,
                                   out=buf.view(torch.float32))
    guard("weights")
    want, tol = definition(q, cache, rows, counts, lse, scale)
    close(out, want, tol)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,H,D,dl,k,n_rows", [
    (1, 1, 32, 16, 1, 3), (1, 20, 320, 256, 512, 4000), (5, 64, 544, 512, 200, 3000),
    (3, 128, 576, 512, 130, 999), (2, 16, 48, 32, 129, 300), (7, 33, 160, 128, 64, 100),
    (2, 129, 192, 128, 257, 700), (1, 1024, 96, 64, 128, 500), (40, 8, 64, 48, 33, 64),
    (1, 256, 576, 512, 300, 5000), (300, 5, 80, 64, 17, 400)])
def test_sizes(dtype, T, H, D, dl, k, n_rows):
    g = gen(T * 1000 + H)
    q, cache, rows, counts = case(g, T, H, D, k, n_rows, dtype)
    out, lse = run(q, cache, rows, counts, dl, 1.0 / math.sqrt(D))
    # what a token's heads give adds up to one, if it sees anything
    total = out.double().sum(1)
    some = torch.isfinite(lse[:, 0])
    assert (total[some] - 1).abs().max() < 1e-3 if some.any() else True
    assert (total[~some] == 0).all()
    run(q, cache, rows, None, dl, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,ld,offset", [(37, 41, 3), (96, 104, 0), (96, 97, 0), (96, 96, 1),
                                         (575, 600, 8), (17, 24, 8), (40, 40, 0), (576, 584, 8)])
def test_layouts(dtype, D, ld, offset):
    """Any width, stride and alignment of cache and queries, strided lists and results."""
    g = gen(D)
    q, cache, rows, counts = case(g, 4, 6, D, 70, 200, dtype, ld=ld, offset=offset)
    dl = max(1, D - 64)
    run(q, cache, rows, counts, dl, 0.1)
    wide = torch.zeros(4, 9, D + 3, dtype=dtype, device=DEV)
    wide[:, 2:8, :D] = q
    strided = wide[:, 2:8, :D]
    assert not strided.is_contiguous()
    lists = torch.full((4, 99), 5, dtype=torch.int32, device=DEV)
    lists[:, 7:77] = rows
    _, lse = satk.latent_attend_rows(q, cache, rows, counts=counts, latent_dim=dl, scale=0.1)
    out = torch.full((4, 80), -3.0, device=DEV)
    satk.latent_rows_weights(strided, cache, lists[:, 7:77], lse, scale=0.1, counts=counts, out=out)
    want, tol = definition(q, cache, rows, counts, lse, 0.1)
    close(out[:, :70], want, tol)
    assert (out[:, 70:] == -3.0).all()
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=0.1, counts=counts, k=33)
    want, tol = definition(q, cache, rows[:, :33].contiguous(),
                           counts.clamp(max=33), lse, 0.1)
    assert out.shape == (4, 33)
    close(out, want, tol)


@pytest.mark.parametrize("D", [96, 35])
def test_bad_rows_and_odd_values(D):
    g = gen(21)
    q, cache, rows, _ = case(g, 3, 16, D, 140, 300, BF16, counts=False)
    rows[0, 3], rows[1, 139], rows[2, 0] = 300, 2**31 - 1, -2**31
    status = i32([0])
    lse = torch.randn(3, 16, generator=g, device=DEV) + 4
    lse[1, 2:5] = -math.inf
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=0.2, status=status)
    assert int(status.item()) == satk.STATUS_BAD_ROW
    want, tol = definition(q, cache, rows, None, lse, 0.2)
    close(out, want, tol)
    assert out[0, 3] == 0 and out[1, 139] == 0 and out[2, 0] == 0
    # a row that is not finite reaches its own entries only; hidden ones nothing
    cache[7] = math.nan
    cache[9, 3] = math.inf
    rows = torch.where((rows == 7) | (rows == 9), 8, rows)
    rows[:, 50] = 7
    rows[:, 60] = 9
    rows[0, 100:] = 7
    counts = i32([100, 140, 140])
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=0.2, counts=counts)
    assert torch.isnan(out[:, 50]).all() and (out[0, 100:] == 0).all()
    clean = cache.clone()
    clean[7], clean[9] = 0, 0
    want, tol = definition(q, clean, rows, counts, lse, 0.2)
    keep = [j for j in range(140) if j not in (50, 60)]
    close(out[:, keep], want[:, keep], tol[:, keep])
    # a NaN of a token's own
    q[1, 7, 0] = math.nan  # (of a head that saw something)
    out = satk.latent_rows_weights(q, clean, rows, lse, scale=0.2)
    assert torch.isnan(out[1][rows[1] >= 0][:50]).all()
    assert torch.isfinite(out[0][rows[0] < 300]).all() and torch.isfinite(out[2]).all()


@pytest.mark.parametrize("scale", [-0.15, 0.0, 1e30])
def test_scales_of_any_sign_and_size(scale):
    g = gen(22)
    q, cache, rows, counts = case(g, 3, 20, 64, 100, 200, BF16)
    _, lse = satk.latent_attend_rows(q, cache, rows, counts=counts, latent_dim=32, scale=scale)
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=scale, counts=counts)
    if scale < 1:
        close(out, *definition(q, cache, rows, counts, lse, scale))
    assert ((out >= 0) & (out <= 1.0 + 1e-5)).all()


def test_empty_calls():
    g = gen(23)
    q, cache, rows, _ = case(g, 3, 4, 64, 10, 20, BF16, counts=False)
    lse = torch.zeros(3, 4, device=DEV)
    assert satk.latent_rows_weights(q[:0], cache, rows[:0], lse[:0], scale=1.0).shape == (0, 10)
    out = satk.latent_rows_weights(q, cache[:0], rows * 0 - 1, lse, scale=1.0)
    assert (out == 0).all()
    out = satk.latent_rows_weights(q, cache, rows, lse, scale=1.0, counts=i32([0, 0, 0]))
    assert (out == 0).all()


def test_offsets_beyond_32_bits():
    g = gen(24)
    ld = 1 << 20
    buf = torch.zeros(3000 * ld, dtype=BF16, device=DEV)
    cache = buf.view(3000, ld)[:, :96]
    cache[2990:] = torch.randn(10, 96, generator=g, device=DEV).to(BF16)
    q = torch.randn(2, 16, 96, generator=g, device=DEV).to(BF16)
    rows = i32([np.arange(2990, 3000), np.arange(2999, 2989, -1)])
    run(q, cache, rows, None, 64, 0.1)


@pytest.mark.parametrize("H,D", [(128, 576), (128, 544), (112, 576), (120, 512), (96, 576), (64, 544),
                                 (256, 320), (16, 64)])
def test_no_wait_is_given_up(H, D):
    """Rings of four panels and more, units of every length: a call takes far less
    than a wait that is given up (two seconds)."""
    g = gen(26)
    T, k = 200, 700
    q, cache, rows, counts = case(g, T, H, D, k, 1000, BF16)
    lse = torch.full((T, H), 9.0, device=DEV)
    status = i32([0])
    call = lambda: satk.latent_rows_weights(q, cache, rows, lse, scale=0.04, counts=counts,  # noqa: E731
                                            status=status)
    first = call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    again = call()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 500 and int(status.item()) == 0
    assert torch.equal(first, again) and torch.isfinite(first).all()


def test_streams_graphs_and_the_same_bits():
    g = gen(25)
    q, cache, rows, counts = case(g, 9, 48, 320, 300, 2000, BF16)
    want, lse = run(q, cache, rows, counts, 256, 0.06)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = satk.latent_rows_weights(q, cache, rows, lse, scale=0.06, counts=counts)
    b = satk.latent_rows_weights(q, cache, rows, lse, scale=0.06, counts=counts)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        satk.latent_rows_weights(q, cache, rows, lse, scale=0.06, counts=counts, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    q = torch.zeros(4, 2, 64, dtype=BF16, device=DEV)
    cache = torch.zeros(9, 64, dtype=BF16, device=DEV)
    rows, lse = torch.zeros(4, 8, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(cache=cache[:, :63]), dict(cache=cache.half()),
               dict(rows=rows.long()), dict(rows=rows[:3]), dict(lse=lse[:3]), dict(lse=lse.half()),
               dict(scale=math.nan), dict(scale=math.inf), dict(k=9), dict(k=0),
               dict(counts=rows[:3, 0].contiguous()), dict(out=torch.zeros(4, 7, device=DEV)),
               dict(out=torch.zeros(4, 8, dtype=BF16, device=DEV)), dict(status=lse),
               dict(q=torch.zeros(4, 2, 577, dtype=BF16, device=DEV),
                    cache=torch.zeros(9, 577, dtype=BF16, device=DEV)),
               dict(q=torch.zeros(4, 1025, 64, dtype=BF16, device=DEV),
                    lse=torch.zeros(4, 1025, device=DEV))):
        args = dict(q=q, cache=cache, rows=rows, lse=lse, scale=1.0)
        with pytest.raises(satk.SatkError):
            satk.latent_rows_weights(**{**args, **kw})
