"""latent_attend_expanded_grad against its definition in 64 bits.

Tolerances, with u half a step of the element type (bf16 2^-8, fp16 2^-11):
  P is off by e = u + ds + (|score| + |lse| + 2) 2^-21 of itself: its rounding, its
    score (fp32 sums of D products: D 2^-23 scale sum |q||k|), its exponent;
  dS likewise, and by P (dv 2^-23 (sum |dout||v| + sum |dout||out|) + |dlse| 2^-22)
    from the two sums whose difference it takes;
    (of calls of up to 16 tokens a request on average, of requests of one tile of
    tokens: two roundings, the second of what the first left, so u^2 for u)
  with fp16 both lose what is below 2^-25;
  the products' n terms are summed in 32 bits (n 2^-23 of the terms' sizes), the
    tail's over the heads too; a result is rounded once (u of itself, fp16 2^-25)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from guards import guarded
from test_gpu_latent import BF16, DEV, F16, U, gen, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


class Case:
    """Inputs of one call: requests of the given new tokens and contexts, causal
    unless row ends are set afterwards."""

    def __init__(self, g, dtype, H, dn, dr, dv, new, context, dlse=False, spare=(0, 0)):
        def normal(*shape):
            return torch.randn(*shape, generator=g, device=DEV).to(dtype)
        keys = [n + c for n, c in zip(new, context)]
        T, S = sum(new) + spare[0], sum(keys) + spare[1]
        self.q, self.k, self.v = normal(T, H, dn + dr), normal(S, H, dn), normal(S, H, dv)
        self.tail = normal(S, dr) if dr else None
        self.dout = normal(T, H, dv)
        self.dlse = torch.randn(T, H, generator=g, device=DEV) if dlse else None
        self.ts, self.ks = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(keys)])
        ends = [c + np.arange(1, n + 1) for n, c in zip(new, context)] + [np.zeros(spare[0])]
        self.ends = i32(np.concatenate(ends))
        self.scale = 1.2 / math.sqrt(dn + dr)

    def starts(self):
        return i32(self.ts), i32(self.ks)

    def forward(self):
        self.out, self.lse = satk.latent_attend_expanded(
            self.q, self.k, self.tail, self.v, *self.starts(), self.ends, scale=self.scale)

    def grad(self, **kw):
        return satk.latent_attend_expanded_grad(
            self.dout, self.q, self.k, self.tail, self.v, self.out, self.lse, *self.starts(),
            self.ends, scale=self.scale, dlse=self.dlse, **kw)


def definition(c, roundings=1):
    """Gradients and tolerances in 64 bits, a request and a head at a time."""
    T, H, D = c.q.shape
    S, _, dn = c.k.shape
    dv, u = c.v.shape[2], U[c.q.dtype]
    tiny = 2.0**-25 if c.q.dtype == F16 else 0.0

    def zeros(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device=DEV)
    dq, tq, gk, tk, gv, tv = (zeros(*x.shape) for x in (c.q, c.q, c.k, c.k, c.v, c.v))
    gt, tt = zeros(S, D - dn), zeros(S, D - dn)
    size_t = zeros(S, D - dn)
    for r in range(len(c.ts) - 1):
        a, b, lo, hi = int(c.ts[r]), int(c.ts[r + 1]), int(c.ks[r]), int(c.ks[r + 1])
        if a == b or lo == hi:
            continue
        seen = torch.arange(hi - lo, device=DEV)[None] < c.ends[a:b, None]
        seen = seen & ~torch.isneginf(c.lse[a:b]).any(1, keepdim=True)
        for h in range(H):
            q, do, o = (x[a:b, h].double() for x in (c.q, c.dout, c.out))
            key = c.k[lo:hi, h].double()
            if c.tail is not None:
                key = torch.cat([key, c.tail[lo:hi].double()], 1)
            val, L = c.v[lo:hi, h].double(), c.lse[a:b, h, None].double()
            L = torch.where(torch.isinf(L), 0.0, L)
            x = q @ key.T * c.scale
            p = torch.where(seen, torch.exp(torch.clamp(x - L, max=0.0)), 0.0)
            delta = (do * o).sum(1, keepdim=True)
            sums = (do.abs() @ val.abs().T + (do * o).abs().sum(1, keepdim=True)) * dv * 2.0**-23
            if c.dlse is not None:
                delta = delta - c.dlse[a:b, h, None].double()
                sums = sums + c.dlse[a:b, h, None].double().abs() * 2.0**-22
            ds = p * (do @ val.T - delta)
            e = u**roundings + (q.abs() @ key.abs().T) * abs(c.scale) * D * 2.0**-23 \
                + (x.abs() + L.abs() + 2) * 2.0**-21
            e_p = torch.where(seen, p * e + tiny, 0.0)
            e_s = torch.where(seen, ds.abs() * e + p * sums + tiny, 0.0)
            n_t, n_k = (b - a) * 2.0**-23, (hi - lo) * 2.0**-23
            s = abs(c.scale)
            gv[lo:hi, h] = p.T @ do
            tv[lo:hi, h] = (e_p + p * n_t).T @ do.abs()
            full = ds.T @ q * c.scale
            t_full = (e_s + ds.abs() * n_t).T @ q.abs() * s
            gk[lo:hi, h], tk[lo:hi, h] = full[:, :dn], t_full[:, :dn]
            gt[lo:hi] += full[:, dn:]
            tt[lo:hi] += t_full[:, dn:]
            size_t[lo:hi] += full[:, dn:].abs()
            dq[a:b, h] = ds @ key * c.scale
            tq[a:b, h] = (e_s + ds.abs() * n_k) @ key.abs() * s
    tt += size_t * H * 2.0**-24
    out = []
    for x, t in ((dq, tq), (gk, tk), (gt, tt), (gv, tv)):
        out.append((x, t + u * x.abs() + tiny + 1e-30))
    return out


def close(got, want, what):
    for name, x, (y, tol) in zip(("dq", "dk", "dtail", "dv"), got, want):
        if x is None:
            assert y.numel() == 0
            continue
        off = (x.double() - y).abs() - tol
        if off.numel() == 0:
            continue
        assert not torch.isnan(off).any(), f"{what} {name}: NaN"
        assert off.max().item() <= 0, f"{what} {name}: beyond the tolerance by {off.max().item():.3g}"


SHAPES = [  # H, dn, dr, dv, new, context
    (1, 16, 0, 16, [1], [0]),
    (3, 64, 32, 64, [5, 1, 70], [0, 9, 0]),
    (2, 128, 64, 128, [300], [0]),
    (2, 128, 64, 128, [129, 64, 1, 200], [31, 700, 128, 0]),
    (5, 96, 48, 80, [64, 63, 65], [1, 0, 64]),
    (2, 192, 64, 128, [200, 33], [100, 0]),
    (1, 256, 0, 128, [150], [150]),
    (4, 32, 16, 112, [1] * 40, [3 * i for i in range(40)]),
    (1, 128, 0, 128, [1], [3000]),
    (2, 80, 64, 96, [700], [60]),
    (1, 208, 48, 16, [140, 260], [0, 1]),
    (9, 48, 64, 32, [257, 127], [0, 129]),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dlse", [False, True])
def test_shapes(dtype, shape, dlse):
    c = Case(gen(shape), dtype, *SHAPES[shape], dlse=dlse)
    c.forward()
    close(c.grad(), definition(c), "shapes")


FEW = [  # H, dn, dr, dv, new, context
    (1, 16, 0, 16, [1], [0]),
    (3, 64, 32, 64, [5, 1, 16], [0, 9, 0]),
    (2, 128, 64, 128, [2, 3, 8], [0, 400, 1100]),
    (16, 128, 64, 128, [4], [0]),
    (5, 96, 48, 80, [64, 1, 1, 0, 1, 0], [130, 0, 64, 0, 127, 3]),
    (2, 192, 64, 128, [7, 0, 33], [100, 0, 0]),
    (1, 256, 0, 128, [16], [150]),
    (2, 80, 64, 96, [8] * 9, [0, 1, 56, 120, 121, 249, 500, 0, 0]),
    (1, 64, 0, 64, [1, 2], [3000, 0]),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", range(len(FEW)))
def test_few_tokens(dtype, shape):
    """P and dS as two operands each."""
    c = Case(gen(100 + shape), dtype, *FEW[shape], dlse=bool(shape & 1))
    c.forward()
    close(c.grad(), definition(c, roundings=2), "few tokens")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_few_tokens_beside_many(dtype):
    """A long request in a call that has few tokens a request on average, and what a
    call of both kinds has in infinities: a weight of 1 whose rest is 0."""
    new = [300] + [1] * 30
    c = Case(gen(120), dtype, 2, 64, 32, 64, new, [40] + [5 * i for i in range(30)], dlse=True)
    assert sum(new) <= 16 * len(new)
    c.forward()
    got, again = c.grad(), c.grad()
    close(got, definition(c), "few beside many")
    for x, y in zip(got, again):
        assert torch.equal(x, y)
    c.dout[310] = math.inf
    got = c.grad()
    assert not torch.isfinite(got[0][310]).any()
    others = torch.arange(len(c.q), device=DEV) != 310
    for x, y in zip(got[:1], again[:1]):
        assert torch.equal(x[others], y[others])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,dn,dr,dv", [(2, 17, 0, 5), (3, 33, 7, 65), (1, 250, 6, 127), (2, 8, 8, 8),
                                        (2, 64, 33, 64), (1, 100, 100, 20)])
def test_odd_widths(dtype, H, dn, dr, dv):
    c = Case(gen(dn), dtype, H, dn, dr, dv, [70, 3, 40], [0, 10, 90], dlse=True)
    c.forward()
    close(c.grad(), definition(c), "odd widths")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dr", [0, 32])
def test_masks(dtype, dr):
    """Row ends in any order, none, one, all and past the keys; keys that no token
    sees; tokens and keys of no request."""
    g = gen(31)
    c = Case(g, dtype, 2, 64, dr, 64, [200, 130, 90, 7], [0, 300, 2, 0], spare=(70, 150))
    rng = np.random.RandomState(31)
    ends = c.ends.cpu().numpy()
    ends[:200] = rng.randint(-2, 230, 200)
    ends[40:120] = 0
    ends[200:330] = rng.choice([1, 64, 128, 129, 257, 10**9], 130)
    ends[330:420] = 0
    ends[427:] = 500
    c.ends = i32(ends)
    c.ks[-1] = c.ks[-2]  # the last request has no keys
    c.forward()
    got = c.grad()
    close(got, definition(c), "masks")
    dq, dk, dtail, dv = got
    assert (dq[420:] == 0).all() and (dq[330:420] == 0).all()
    n = int(c.ks[-1])
    assert (dk[n:] == 0).all() and (dv[n:] == 0).all()
    if dr:
        assert (dtail[n:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dn,dr,dv", [(64, 32, 64), (33, 5, 20), (128, 64, 128)])
def test_what_is_not_seen_may_be_anything(dtype, dn, dr, dv):
    """NaN and infinities in rows that a token does not see, in tokens that see
    nothing and in rows of no request reach no other gradient."""
    g = gen(32)
    c = Case(g, dtype, 2, dn, dr, dv, [150, 100], [40, 0], dlse=True, spare=(20, 30))
    rng = np.random.RandomState(32)
    ends = c.ends.cpu().numpy()
    ends[[3, 70, 149]] = 0
    ends[:150] = np.minimum(ends[:150], 170)  # keys 170.. of the first request: unseen
    ends[150:250] = rng.randint(0, 60, 100)
    c.ends = i32(ends)
    blind = [t for t in range(250) if ends[t] <= 0] + list(range(250, 270))
    unseen = list(range(170, 190)) + list(range(190 + 60, 290)) + list(range(290, 320))
    for x in (c.q, c.dout):
        x[blind] = 0
    for x in (c.k, c.v, c.tail):
        x[unseen] = 0
    c.forward()
    want = definition(c)
    clean = c.grad()
    close(clean, want, "clean")
    for i, t in enumerate(blind):
        c.q[t, i % 2, i % 5] = (math.nan, math.inf, -math.inf)[i % 3]
        c.dout[t, :, i % 3] = (math.inf, math.nan)[i % 2]
        c.dlse[t] = math.nan
    c.out[blind] = math.nan
    for i, s in enumerate(unseen):
        c.k[s, i % 2, i % 7] = (math.nan, math.inf)[i % 2]
        c.v[s, :, i % 3] = (math.inf, math.nan)[i % 2]
        c.tail[s, i % 5] = math.nan
    got = c.grad()
    close(got, want, "not seen")
    for x, y in zip(got, clean):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dn,dr,dv", [(64, 32, 64), (40, 3, 24)])
def test_rows_that_are_not_finite_reach_what_they_should(dn, dr, dv):
    """A key that is not finite makes the tokens that see it not finite (in its own head)
    and no other; a token that is not finite makes the keys that it sees NaN."""
    c = Case(gen(33), BF16, 2, dn, dr, dv, [200], [0])
    c.forward()
    want = definition(c)
    keep = c.k[100, 1, 2].clone()
    c.k[100, 1, 2] = math.inf
    dq, dk, dtail, _ = c.grad()
    assert (~torch.isfinite(dq[100:, 1])).any(1).all()  # (a weight times infinity, or NaN)
    close((dq[:100], dk[:, 0]), ([x[:100] for x in want[0]], [x[:, 0] for x in want[1]]), "key")
    close((dq[:, 0],), ([x[:, 0] for x in want[0]],), "other head")
    c.k[100, 1, 2] = keep
    c.dout[60, 0, 1] = math.nan
    dq, dk, dtail, dv_ = c.grad()
    assert torch.isnan(dv_[:61, 0]).any(1).all() and torch.isnan(dk[:61, 0]).any(1).all()
    assert torch.isnan(dq[60, 0]).any()
    for x, y in ((dv_[61:], want[3]), (dk[61:], want[1])):
        close((x,), ([z[61:] for z in y],), "token")
    close((dv_[:, 1],), ([z[:, 1] for z in want[3]],), "other head")
    others = [t for t in range(200) if t != 60]
    close((dq[others],), ([z[others] for z in want[0]],), "other tokens")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pad", [8, 3])
def test_layouts(dtype, pad):
    """Strided inputs and gradients (aligned and not), guards around those, and the
    memory between their rows."""
    g = gen(34)
    c = Case(g, dtype, 3, 64, 16, 48, [90, 140], [30, 0], dlse=True)
    c.forward()
    want = definition(c)

    def strided(x):
        shape = list(x.shape)
        wide = torch.full([shape[0] + 1] + [s + pad for s in shape[1:]], 5.0, dtype=x.dtype, device=DEV)
        view = wide[1:, 1:-1 * (pad - 1), :shape[2]][:, :shape[1]] if len(shape) == 3 else wide[1:, :shape[1]]
        view.copy_(x)
        return view
    for name in ("q", "k", "v", "tail", "dout", "out"):
        setattr(c, name, strided(getattr(c, name)))
    grads = {}
    for name, like in (("dq", c.q), ("dk", c.k), ("dtail", c.tail), ("dv", c.v)):
        shape = list(like.shape)
        wide = torch.full([shape[0]] + shape[1:-1] + [shape[-1] + pad], 7.0, dtype=dtype, device=DEV)
        grads[name] = (wide[..., :shape[-1]], wide)
    size = satk.latent_expanded_grad_workspace_bytes(len(c.q), len(c.k), 2, 3, 16)
    buf, guard = guarded(((size + 3) // 4,), torch.int32)
    got = c.grad(workspace=buf, **{n: x for n, (x, _) in grads.items()})
    guard("workspace")
    close(got, want, "layouts")
    for name, (x, wide) in grads.items():
        assert (wide[..., x.shape[-1]:] == 7).all(), name


def test_gradient_against_differences():
    """Along random directions, against differences of the definition's forward pass
    in 64 bits."""
    g = gen(35)
    c = Case(g, F16, 2, 48, 16, 32, [60, 33], [20, 0], dlse=True)
    c.forward()
    got = c.grad()

    def loss(q, k, tail, v):
        total = 0.0
        for r in range(2):
            a, b, lo, hi = c.ts[r], c.ts[r + 1], c.ks[r], c.ks[r + 1]
            hide = torch.arange(int(hi - lo), device=DEV)[None] >= c.ends[a:b, None]
            for h in range(2):
                key = torch.cat([k[lo:hi, h], tail[lo:hi]], 1)
                x = (q[a:b, h] @ key.T * c.scale).masked_fill(hide, -math.inf)
                lse = torch.logsumexp(x, 1)
                o = torch.exp(x - lse[:, None]) @ v[lo:hi, h]
                total = total + (o * c.dout[a:b, h].double()).sum() \
                    + (lse * c.dlse[a:b, h].double()).sum()
        return total
    at = [x.double() for x in (c.q, c.k, c.tail, c.v)]
    want = definition(c)
    for i in range(4):
        way = torch.randn(at[i].shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-5
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + h * way, at[i] - h * way
        slope = (loss(*plus) - loss(*minus)) / (2 * h)
        # out's rounding enters through delta: u of each |dout||out| times the weights' pull
        tol = (want[i][1] * way.abs()).sum() + 4 * U[F16] * (want[i][0].abs() * way.abs()).sum()
        assert ((got[i].double() * way).sum() - slope).abs() <= tol


def test_definition_is_the_gradient():
    """The 64-bit definition against torch's own differentiation of the forward pass
    in 64 bits, out and lse exact."""
    c = Case(gen(36), BF16, 2, 32, 16, 32, [40], [9], dlse=True)
    q, k, tail, v = (x.double().requires_grad_() for x in (c.q, c.k, c.tail, c.v))
    hide = torch.arange(49, device=DEV)[None] >= c.ends[:, None]
    key = torch.cat([k, tail[:, None].expand(-1, 2, -1)], 2)
    x = torch.einsum("thd,shd->hts", q, key) * c.scale
    x = x.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(x, 2)
    out = torch.einsum("hts,shd->thd", torch.exp(x - lse[..., None]), v)
    ((out * c.dout.double()).sum() + (lse.T * c.dlse.double()).sum()).backward()
    c.out, c.lse = out.detach(), lse.T.detach().contiguous()
    for (mine, _), x in zip(definition(c), (q, k, tail, v)):
        assert (mine - x.grad).abs().max() <= 1e-12 * x.grad.abs().max()


def test_offsets_beyond_32_bits():
    g = gen(37)
    c = Case(g, BF16, 1, 64, 16, 64, [3], [0])
    c.forward()
    want = definition(c)
    ld = (1 << 30) + 16

    def far(x):
        buf = torch.zeros(2 * ld + 256, dtype=BF16, device=DEV)
        y = buf.as_strided(x.shape, (ld,) + (x.shape[-1],) * (x.dim() - 2) + (1,))
        y.copy_(x)
        return y
    for name in ("q", "k", "v", "tail", "dout", "out"):
        setattr(c, name, far(getattr(c, name)))
    close(c.grad(dq=far(c.q), dk=far(c.k), dtail=far(c.tail), dv=far(c.v)), want, "far")


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e30])
def test_scales_of_any_sign_and_size(scale):
    c = Case(gen(38), BF16, 2, 64, 0, 64, [140], [0])
    c.scale = scale
    c.forward()
    got = c.grad()
    if abs(scale) < 1:
        close(got, definition(c), "scale")
    # at any size the weights are within [0, 1]: |dv| <= sum |dout|
    assert (got[3].double().abs() <= c.dout.double().abs().sum(0) * (1 + 2.0**-7)).all()


def test_many_requests():
    rng = np.random.RandomState(39)
    new = rng.randint(0, 5, 300)
    new[[7, 150]] = 200, 130
    ctx = rng.randint(0, 40, 300)
    c = Case(gen(39), BF16, 2, 32, 16, 32, list(new), list(ctx))
    c.forward()
    close(c.grad(), definition(c), "many requests")


def test_no_requests_no_tokens_no_keys():
    g = gen(40)
    c = Case(g, BF16, 2, 32, 16, 32, [10], [5])
    c.forward()
    c.ts, c.ks = np.array([0]), np.array([0])
    for x in c.grad():
        assert (x == 0).all()
    c = Case(g, BF16, 2, 32, 16, 32, [0], [5])
    c.forward()
    dq, dk, dtail, dv = c.grad()
    assert dq.shape[0] == 0 and (dk == 0).all() and (dtail == 0).all() and (dv == 0).all()
    c = Case(g, BF16, 2, 32, 16, 32, [6], [0])
    c.k, c.v, c.tail, c.ks = c.k[:0], c.v[:0], c.tail[:0], np.array([0, 0])
    c.forward()
    dq, dk, dtail, dv = c.grad()
    assert (dq == 0).all() and dk.shape[0] == dv.shape[0] == dtail.shape[0] == 0


@pytest.mark.parametrize("shape", [(2, 128, 64, 128, [300, 77], [100, 0]), (2, 33, 3, 20, [50], [9])])
def test_streams_graphs_and_the_same_bits(shape):
    c = Case(gen(41), BF16, *shape)
    c.forward()
    want = c.grad()
    close(want, definition(c), "first")
    torch.cuda.synchronize()
    results = []
    for _ in range(3):
        with torch.cuda.stream(torch.cuda.Stream()):
            results.append(c.grad())
    torch.cuda.synchronize()
    into = {n: torch.empty_like(x) for n, x in zip(("dq", "dk", "dtail", "dv"), want)}
    starts = c.starts()
    size = satk.latent_expanded_grad_workspace_bytes(len(c.q), len(c.k), len(c.ts) - 1, shape[0], shape[2])
    workspace = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:  # two graphs that share a workspace, one after the other
        with torch.cuda.graph(graph):
            satk.latent_attend_expanded_grad(c.dout, c.q, c.k, c.tail, c.v, c.out, c.lse, *starts,
                                             c.ends, scale=c.scale, workspace=workspace, **into)
    for graph in graphs + graphs[:1]:
        for x in into.values():
            x.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        results.append(tuple(x.clone() for x in into.values()))
    for r in results:
        for x, y in zip(r, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dn,dr,dv", [(128, 64, 128), (256, 0, 128), (192, 64, 64), (208, 48, 128), (64, 0, 64),
                                      (16, 16, 16), (144, 64, 112)])
def test_no_wait_is_given_up(dtype, dn, dr, dv):
    """A call over many tiles takes far less than a wait that is given up (two
    seconds)."""
    c = Case(gen(44), dtype, 3, dn, dr, dv, [700, 3, 260], [500, 40, 0])
    c.forward()
    first = c.grad()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    again = c.grad()
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 500
    for x, y in zip(first, again):
        assert x is None or (torch.equal(x, y) and torch.isfinite(x).all())


@pytest.mark.parametrize("shape", [3, 5, 9])
def test_calls_in_a_row_with_cold_caches(shape):
    """The same bits whatever the memory system makes of the order in which loads,
    products and rows' checks arrive: caches full of NaN patterns in between."""
    c = Case(gen(43), BF16, *SHAPES[shape])
    c.forward()
    want = c.grad()
    close(want, definition(c), "first")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for i in range(40):
        if i % 2:
            flush.fill_(255)
        for x, y in zip(c.grad(), want):
            assert torch.equal(x, y), i


def test_refusals():
    c = Case(gen(42), BF16, 2, 32, 16, 32, [10], [5])
    c.forward()
    ok = dict(dout=c.dout, q=c.q, k=c.k, tail=c.tail, v=c.v, out=c.out, lse=c.lse,
              token_starts=c.starts()[0], key_starts=c.starts()[1], row_ends=c.ends, scale=0.1)
    size = satk.latent_expanded_grad_workspace_bytes(10, 15, 1, 2, 16)
    for kw in (dict(dout=c.dout.float()), dict(dout=c.dout[:9]), dict(q=c.q[:, :, :47]),
               dict(k=c.k[:, :1]), dict(k=c.k.half()), dict(v=c.v[:14]), dict(tail=c.tail[:14]),
               dict(tail=c.tail[:, :15]), dict(tail=None), dict(out=c.out[:, :, :31]),
               dict(out=c.out.half()), dict(lse=c.lse[:9]), dict(lse=c.lse.double()),
               dict(token_starts=c.ends[:0]), dict(key_starts=c.ends[:1]),
               dict(row_ends=c.ends[:9]), dict(row_ends=c.ends.long()), dict(scale=math.nan),
               dict(dlse=c.lse[:, :1]), dict(dlse=c.lse.half()), dict(dq=c.q[:9]),
               dict(dk=c.k.half()), dict(dtail=c.tail[:, :8]), dict(dv=c.v[:, :, :8]),
               dict(workspace=torch.empty(size - 1, dtype=torch.uint8, device=DEV)),
               dict(workspace=torch.empty(size + 16, dtype=torch.uint8, device=DEV)[1:])):
        with pytest.raises(satk.SatkError):
            satk.latent_attend_expanded_grad(**{**ok, **kw})
    with pytest.raises(satk.SatkError, match="dtail without"):
        satk.latent_attend_expanded_grad(**{**ok, "tail": None, "q": c.q[:, :, :32], "dtail": c.tail})
