"""Values at the ends of their ranges in the latent-cache calls: starts beyond
the tokens, scores near the ends of fp32, values that are not finite."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from test_gpu_latent import BF16, DEV, F16, U, expanded_case, expanded_check, gen, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


@pytest.mark.parametrize("dn", [64, 20])  # tensor cores, and the form for any width
@pytest.mark.parametrize("first,last", [(0, 2**31 - 1), (5, 2**31 - 1), (0, 2**31 - 9), (7, 300),
                                        (-2**31, 2**31 - 1)])
def test_expanded_starts_beyond_the_tokens(dn, first, last):
    """A last start past the tokens ends the request at the last token; tokens
    before the first start have empty rows."""
    T, H, dv = 150, 2, 32
    q, k, _, v, _, ks, ends = expanded_case(gen(81), BF16, H, dn, 0, dv, [T], [10])
    guard = torch.full((T + 64, H, dv), 3.0, dtype=BF16, device=DEV)
    lse_guard = torch.full((T + 64, H), 3.0, device=DEV)
    o, lse = satk.latent_attend_expanded(q, k, None, v, i32([first, last]), i32(ks), i32(ends),
                                         scale=0.2, out=guard[32:-32], lse=lse_guard[32:-32])
    begin = max(first, 0)
    assert torch.all(o[:begin] == 0) and torch.all(torch.isneginf(lse[:begin]))
    expanded_check(q, k, None, v, np.array([begin, T]), ks, ends, o, lse, 0.2)
    for x in (guard, lse_guard):
        assert torch.all(x[:32] == 3.0) and torch.all(x[-32:] == 3.0)


def peaks(g, dtype, n, order, level):
    """n keys' factors 1..120 times 2**level (exact in 16 bits) in an order, the
    largest of them on two keys: [n], and the numbers of those two."""
    m = torch.randint(1, 100, (n,), generator=g, device=DEV).double()
    a, b = (0, 1) if order == "first" else (n - 2, n - 1) if order == "last" else (n // 3, n // 2)
    if order == "rising":
        m = torch.arange(n, device=DEV).double() * 100 // n
        a, b = n - 3, n - 2
    m[a] = m[b] = 120
    return (m * 2.0**level).to(dtype), (a, b)


# (type, exponents of key and query): products of 2**20 to 2**120 and beyond what
# a reference of -1e30 would tell from no score at all
LEVELS = [(BF16, 10, 10), (BF16, 20, 13), (BF16, 30, 30), (BF16, 50, 50), (BF16, 60, 57),
          (F16, 8, 14)]


@pytest.mark.parametrize("dtype,key_level,query_level", LEVELS)
@pytest.mark.parametrize("order", ["first", "last", "between", "rising"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("form", ["pages", "rows", "warp", "expanded", "expanded warp"])
def test_scores_of_any_size(form, sign, order, dtype, key_level, query_level):
    """Scores so far apart that a token's two best keys share all its weight:
    its output is the mean of their values.  With the sign turned the smallest
    factors are the best ones; there all keys get one factor and share it."""
    g = gen(83)
    n, T, H, dl, dr, scale = 700, 3, 16, 64, 16, 0.7
    D = dl + dr
    factor, best = peaks(g, dtype, n, order, key_level)
    if sign < 0:
        factor[:] = factor[best[0]]
        best = range(n)
    width = 88 if form != "warp" else 83  # an odd row stride takes the form for any layout
    rows = torch.zeros(n, width, dtype=dtype, device=DEV)[:, :D]
    rows[:, :dl] = torch.randn(n, dl, generator=g, device=DEV)
    rows[:, dl] = factor
    q = torch.zeros(T, H, D, dtype=dtype, device=DEV)
    q[:, :, dl] = sign * 2.0**query_level
    if form == "pages":
        table = i32([range(n // 28)])
        o, lse = satk.latent_attend(q, rows, i32([0] * T), table, i32([n] * T), block_size=28,
                                    stride_rows=28, latent_dim=dl, scale=scale)
        o2, lse2 = satk.latent_attend(q, rows, i32([0] * T), i32([[*range(43), -1]]),
                                      i32([n - n % 16] * T), block_size=16, stride_rows=16,
                                      latent_dim=dl, scale=scale)
    elif form in ("rows", "warp"):
        o, lse = satk.latent_attend_rows(q, rows, i32([range(n)] * T), latent_dim=dl, scale=scale)
    else:
        dn = 32 if form == "expanded" else 20
        k = torch.zeros(n, H, dn, dtype=dtype, device=DEV)
        k[:, :, 3] = factor[:, None]
        qe = torch.zeros(T, H, dn, dtype=dtype, device=DEV)
        qe[:, :, 3] = sign * 2.0**query_level
        v = rows[:, None, :32].expand(n, H, 32).contiguous()
        o, lse = satk.latent_attend_expanded(qe, k, None, v, i32([0, T]), i32([0, n]),
                                             i32([n] * T), scale=scale)

    def check(o, lse, best):
        values = rows[list(best), :o.shape[2]].double()
        want = values.mean(0)
        # the output's rounding and fp32 sums of equal weights
        tol = U[dtype] * want.abs() + 1e-5 * values.abs().mean(0)
        assert ((o.double() - want).abs() <= tol).all()
        top = sign * factor[best[0]].double() * 2.0**query_level * scale + math.log(len(best))
        assert ((lse.double() - top).abs() <= 1e-6 * top.abs()).all()

    check(o, lse, best)
    if form == "pages":
        seen = n - n % 16
        if sign < 0:
            check(o2, lse2, range(seen))
        elif max(best) < seen:
            check(o2, lse2, best)


@pytest.mark.parametrize("new,context", [([40, 3], [0, 90]), ([70], [500])])
def test_causal_chunk_of_far_scores(new, context):
    """The same far below -1e30 where tokens of a group see different keys: the
    first tiles of some columns hold none of their keys."""
    g = gen(85)
    H, dl, D, scale = 8, 64, 80, 0.7
    lens = [a + b for a, b in zip(new, context)]
    width = -(-max(lens) // 16)
    table = np.arange(len(new) * width).reshape(len(new), width)
    rows = torch.zeros(len(new) * width * 16, D, dtype=BF16, device=DEV)
    rows[:, :dl] = torch.randn(rows.shape[0], dl, generator=g, device=DEV)
    rows[:, dl] = 2.0**55
    req = np.repeat(np.arange(len(new)), new)
    ends = np.concatenate([c + 1 + np.arange(n) for c, n in zip(context, new)])
    q = torch.zeros(len(req), H, D, dtype=BF16, device=DEV)
    q[:, :, dl] = -2.0**57
    o, lse = satk.latent_attend(q, rows, i32(req), i32(table), i32(ends), block_size=16,
                                stride_rows=16, latent_dim=dl, scale=scale)
    score = -2.0**112 * scale
    for t, r in enumerate(req):
        v = rows[r * width * 16:][:ends[t], :dl].double()
        assert ((o[t].double() - v.mean(0)).abs()
                <= U[BF16] * v.mean(0).abs() + 1e-5 * v.abs().mean(0)).all()
        assert ((lse[t].double() - score).abs() <= 1e-6 * abs(score)).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dn", [64, 20])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_expanded_lse_goes_by_the_keys_alone(what, dn, dtype):
    """Values that are not finite, in tiles that every token sees whole and in
    those that only some see: the lse of every token is that of its scores, and
    only the outputs of tokens that see them are not finite."""
    g = gen(87)
    H, dv, T, context = 2, 32, 200, 300
    q, k, _, v, ts, ks, ends = expanded_case(g, dtype, H, dn, 0, dv, [T], [context])
    for key in (70, 330, 421):
        clean, _ = satk.latent_attend_expanded(q, k, None, v, i32(ts), i32(ks), i32(ends),
                                               scale=0.2)
        odd = v.clone()
        odd[key, 1, 7] = what
        o, lse = satk.latent_attend_expanded(q, k, None, odd, i32(ts), i32(ks), i32(ends),
                                             scale=0.2)
        for t in range(T):
            s = torch.einsum("hd,nhd->hn", q[t].double(), k[:ends[t]].double()) * 0.2
            want = torch.logsumexp(s, 1)
            ds = torch.einsum("hd,nhd->hn", q[t].double().abs(),
                              k[:ends[t]].double().abs()).amax(1) * 0.2 * dn * 2.0**-23
            assert ((lse[t].double() - want).abs() <= ds + 1e-5 + 1e-6 * want.abs()).all(), t
            assert torch.equal(o[t, 0], clean[t, 0])
            if ends[t] > key:
                assert not torch.isfinite(o[t, 1, 7])
            else:
                assert torch.equal(o[t, 1], clean[t, 1])
