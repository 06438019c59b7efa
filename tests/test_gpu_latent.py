"""The latent-cache operators against their definitions in 64 bits.

Tolerances are derived from the roundings an implementation may make: u is
half a step of the element type (bf16 2^-8, fp16 2^-11).  An attention output
differs from the definition by at most
    u |out|                       the output's rounding
  + u sum_j p_j |v_j|             the weights' rounding before the product
  + 2 ds sum_j p_j |v_j|          scores off by ds (fp32 sums of D products:
                                  D 2^-23 scale sum |q||k|), in numerator and
                                  denominator
  + 1e-5 sum_j p_j |v_j|          exp2, the joins and the division in 32 bits
  + N 2^-25 max|v| (fp16 only)    weights below fp16's smallest step, relative
                                  to a largest weight of at least 1
and its lse by ds + 1e-5 + 1e-6 |lse|."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from guards import guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F16 = torch.bfloat16, torch.float16
U = {BF16: 2.0**-8, F16: 2.0**-11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


def guarded16(shape, dtype):
    """A guarded 16-bit buffer: the int32 guards of an allocation around it."""
    n = int(np.prod(shape))
    inner, check = guarded(((n + 1) // 2,), torch.int32)
    return inner.view(dtype)[:n].view(*shape), check


def one_token(q, keys, dv, scale, u):
    """softmax attention of q [H, D] over keys [N, D] (values: the first dv
    columns) in 64 bits, and the elementwise tolerance of out and lse."""
    q, keys = q.double(), keys.double()
    H = q.shape[0]
    if keys.shape[0] == 0:
        z = torch.zeros(H, dv, dtype=torch.float64, device=DEV)
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device=DEV), z, z[:, 0]
    return attention64(q, keys, keys[:, :dv], scale, u)


def attention64(q, keys, v, scale, u):
    """q [H, D] over keys [N, D] or [H, N, D], v likewise."""
    eq = "hd,nd->hn" if keys.dim() == 2 else "hd,hnd->hn"
    ev = "hn,nd->hd" if v.dim() == 2 else "hn,hnd->hd"
    s = torch.einsum(eq, q, keys) * scale
    ds = torch.einsum(eq, q.abs(), keys.abs()).amax(1) * abs(scale) * q.shape[1] * 2.0**-23
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out, mass = torch.einsum(ev, p, v), torch.einsum(ev, p, v.abs())
    tol = u * out.abs() + (u + 2 * ds[:, None] + 1e-5) * mass
    if u == U[F16]:
        tol = tol + keys.shape[-2] * 2.0**-25 * v.abs().max() + 2.0**-25
    return out, lse, tol, ds + 1e-5 + 1e-6 * lse.abs()


def assert_close(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite places differ"
    f = torch.isfinite(want)
    assert torch.equal(torch.isneginf(got), torch.isneginf(want)), what
    off = (got - want).abs() - tol
    worst = off[f].max().item() if f.any() else 0.0
    assert worst <= 0, f"{what}: beyond the tolerance by {worst:.3g}"


def latent_rows(g, rows, D, dtype, ld=None, offset=0):
    """Cache [rows, D] with row stride ld, its base `offset` elements into an
    allocation, holding standard normal values on a shared direction."""
    ld = D if ld is None else ld
    buf = torch.zeros(rows * ld + offset + 8, dtype=dtype, device=DEV)
    cache = buf[offset:offset + rows * ld].view(rows, ld)[:, :D]
    cache.copy_(torch.randn(rows, D, generator=g, device=DEV)
                + 0.5 * torch.randn(D, generator=g, device=DEV))
    return cache


class Paged:
    """Requests with paged caches of the given lengths (drafted tokens
    included) in shuffled blocks; rows that hold no token are NaN."""

    def __init__(self, g, rng, lens, D, block, dtype, stride_rows=None, **layout):
        self.block, self.stride = block, stride_rows or block
        width = max(1, max(-(-n // block) for n in lens) + 1)
        ids = rng.permutation(len(lens) * width + 2)[:len(lens) * width]
        self.table = ids.reshape(len(lens), width)
        rows = (len(lens) * width + 2) * self.stride
        self.cache = latent_rows(g, rows, D, dtype, **layout)
        used = torch.zeros(rows, dtype=torch.bool)
        for r, n in enumerate(lens):
            used[self.rows(r, np.arange(n))] = True
        self.cache[~used.to(DEV)] = float("nan")

    def rows(self, r, j):
        j = np.asarray(j, dtype=np.int64)
        return torch.from_numpy(self.table[r, j // self.block] * self.stride + j % self.block)

    def keys(self, r, j):
        return self.cache[self.rows(r, j).to(DEV)]


def run_paged(q, pg, req, ends, dl, scale, tree=None, dtype=BF16, check_guard=True):
    T, H, _ = q.shape
    out, check = guarded16((T, H, dl), dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = satk.latent_attend(q, pg.cache, i32(req), i32(pg.table), i32(ends),
                                block_size=pg.block, stride_rows=pg.stride, latent_dim=dl,
                                scale=scale, tree=tree, out=out, status=status)
    torch.cuda.synchronize()
    check("latent_attend")
    return o, lse, int(status.item())


# (dtype, heads, latent, tail, block, causal ends of one token each)
DECODE = [
    (BF16, 16, 128, 32, 16, [1, 0, 63, 64, 65, 127, 128, 129, 300]),
    (F16, 16, 128, 0, 16, [5, 17, 64, 200]),
    (BF16, 1, 64, 16, 32, [70, 1, 640]),
    (BF16, 5, 48, 48, 64, [33, 100]),
    (F16, 20, 320, 64, 64, [257, 3]),
    (BF16, 64, 512, 64, 64, [500, 64, 65]),
    (BF16, 64, 512, 0, 128, [129]),
    (BF16, 65, 256, 32, 16, [77, 400]),
    (F16, 128, 448, 64, 32, [90, 1]),
    (BF16, 200, 192, 16, 16, [130]),
    (BF16, 32, 384, 64, 64, [5000, 1, 0, 2049]),
    (BF16, 7, 50, 6, 10, [45, 0, 1]),          # widths that no 16-byte access fits
    (F16, 3, 17, 3, 7, [29, 100]),
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_paged_decode(case):
    dtype, H, dl, dr, block, ends = DECODE[case]
    g, rng = gen(100 + case), np.random.RandomState(case)
    D, R = dl + dr, len(ends)
    pg = Paged(g, rng, ends, D, block, dtype, stride_rows=block + (3 if case % 2 else 0))
    q = torch.randn(R, H, D, generator=g, device=DEV).to(dtype)
    scale = 1.3 / math.sqrt(D)
    o, lse, st = run_paged(q, pg, range(R), ends, dl, scale, dtype=dtype)
    assert st == 0
    for t in range(R):
        w = one_token(q[t], pg.keys(t, np.arange(ends[t])), dl, scale, U[dtype])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("dtype,H,dl,dr,ld,offset,q_pad", [
    (BF16, 12, 128, 32, 168, 0, 0), (BF16, 12, 128, 32, 161, 0, 0), (F16, 9, 128, 32, 160, 1, 0),
    (BF16, 16, 128, 64, 192, 8, 5), (F16, 40, 256, 16, 512, 16, 8)])
def test_paged_layouts(dtype, H, dl, dr, ld, offset, q_pad):
    """Row strides and bases of the cache that 16-byte loads fit or do not, and
    queries and outputs with strides of their own, heads before tokens."""
    g, rng = gen(7), np.random.RandomState(7)
    D, ends = dl + dr, [130, 64, 1]
    pg = Paged(g, rng, ends, D, 16, dtype, ld=ld, offset=offset)
    store = torch.randn(H, 3, D + q_pad, generator=g, device=DEV).to(dtype)
    q = store.transpose(0, 1)[..., :D]
    canvas = torch.full((H, 3, dl + 4), -7.0, dtype=dtype, device=DEV)
    out = canvas.transpose(0, 1)[..., :dl]
    _, lse = satk.latent_attend(q, pg.cache, i32(range(3)), i32(pg.table), i32(ends),
                                block_size=16, stride_rows=16, latent_dim=dl, scale=0.1, out=out)
    assert torch.all(canvas[..., dl:] == -7.0)
    for t in range(3):
        w = one_token(q[t], pg.keys(t, np.arange(ends[t])), dl, 0.1, U[dtype])
        assert_close(out[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("dtype,H,new,context", [
    (BF16, 16, [70, 3, 1], [0, 61, 130]), (F16, 4, [33, 64], [500, 0]), (BF16, 128, [5], [64]),
    (BF16, 64, [2, 2, 2], [62, 63, 64]), (BF16, 1, [200], [1])])
def test_paged_chunk(dtype, H, new, context):
    """Several causal tokens a request, and NaN in the tokens after each one's
    end: keys that later tokens see and earlier ones do not."""
    g, rng = gen(9), np.random.RandomState(9)
    dl, D = 128, 160
    lens = [c + n for c, n in zip(context, new)]
    pg = Paged(g, rng, lens, D, 16, dtype)
    req = np.repeat(np.arange(len(new)), new)
    ends = np.concatenate([c + 1 + np.arange(n) for c, n in zip(context, new)])
    q = torch.randn(len(req), H, D, generator=g, device=DEV).to(dtype)
    for bad in (False, True):
        if bad:  # the last token's row of each request
            for r, n in enumerate(lens):
                pg.cache[pg.rows(r, [n - 1]).to(DEV)] = float("inf") if r % 2 else float("nan")
        o, lse, st = run_paged(q, pg, req, ends, dl, 0.1, dtype=dtype)
        assert st == 0
        for t, r in enumerate(req):
            if bad and ends[t] == lens[r]:
                assert not torch.isfinite(o[t]).all()
                continue
            w = one_token(q[t], pg.keys(r, np.arange(ends[t])), dl, 0.1, U[dtype])
            assert_close(o[t], w[0], w[2], f"out, token {t} {bad}")
            assert_close(lse[t], w[1], w[3], f"lse, token {t} {bad}")


def make_tree(rng, n, words):
    bits = np.zeros((n, words), dtype=np.uint32)
    for i in range(n):
        if i:
            bits[i] |= bits[rng.randint(0, i)]
        bits[i, i // 32] |= np.uint32(1 << (i % 32))
    return bits


@pytest.mark.parametrize("dtype,H,new,context", [
    (BF16, 16, [7, 24, 40], [100, 0, 63]), (F16, 2, [64, 33], [128, 5]),
    (BF16, 96, [9], [1000]), (BF16, 16, [6, 6], [0, 0])])
def test_paged_tree(dtype, H, new, context):
    g, rng = gen(11), np.random.RandomState(11)
    dl, D, words = 192, 224, 2
    lens = [c + n for c, n in zip(context, new)]
    pg = Paged(g, rng, lens, D, 16, dtype)
    bits = np.concatenate([make_tree(rng, n, words) for n in new])
    bits[3] = 0  # a token that sees its context alone (nothing, where that is empty)
    req, ends = np.repeat(np.arange(len(new)), new), np.repeat(context, new)
    q = torch.randn(len(req), H, D, generator=g, device=DEV).to(dtype)
    tree = torch.from_numpy(bits.view(np.int32)).to(DEV)
    o, lse, st = run_paged(q, pg, req, ends, dl, 0.1, tree=tree, dtype=dtype)
    assert st == 0
    for t, r in enumerate(req):
        j = list(range(ends[t])) + [ends[t] + b for b in range(64)
                                    if int(bits[t, b // 32]) >> (b % 32) & 1]
        w = one_token(q[t], pg.keys(r, j), dl, 0.1, U[dtype])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


def test_paged_requests_out_of_order_and_shared():
    """Tokens of one request apart from each other, two requests on the same
    blocks, and the same result from a side stream and a graph."""
    g, rng = gen(13), np.random.RandomState(13)
    pg = Paged(g, rng, [200, 90, 200], 96, 16, BF16)
    pg.table[2] = pg.table[0]
    req, ends = [2, 0, 1, 0, 0, 2], [200, 3, 90, 150, 151, 199]
    q = torch.randn(6, 24, 96, generator=g, device=DEV).to(BF16)
    o, lse, _ = run_paged(q, pg, req, ends, 64, 0.2)
    for t, r in enumerate(req):
        w = one_token(q[t], pg.keys(r, np.arange(ends[t])), 64, 0.2, U[BF16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
    args = (q, pg.cache, i32(req), i32(pg.table), i32(ends))
    kw = dict(block_size=16, stride_rows=16, latent_dim=64, scale=0.2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, l2 = satk.latent_attend(*args, **kw)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = satk.latent_attend(*args, **kw)
    q.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    o4, l4 = satk.latent_attend(*args, **kw)
    assert torch.equal(o3, o4) and torch.equal(l3, l4)


def test_paged_bad_pages():
    """Requests outside the table, blocks outside the cache and ends past the
    table: nothing of them is read, the status says so, other tokens keep
    their results."""
    g, rng = gen(15), np.random.RandomState(15)
    pg = Paged(g, rng, [100, 100, 100], 96, 16, BF16)
    good = pg.table.copy()
    pg.table[1, 2] = 10**6   # keys 32..47 of request 1
    req, ends = [0, 1, 2, 3, -1], [100, 100, 10**9, 50, 50]
    q = torch.randn(5, 16, 96, generator=g, device=DEV).to(BF16)
    pg.cache[torch.isnan(pg.cache)] = 0.25  # request 2 reads to its table's end
    o, lse, st = run_paged(q, pg, req, ends, 64, 0.2)
    assert st == satk.STATUS_BAD_REQUEST | satk.STATUS_BAD_ROW
    reach = good.shape[1] * 16
    for t, j in ((0, np.arange(100)), (1, [j for j in range(100) if j // 16 != 2]),
                 (2, np.arange(reach)), (3, []), (4, [])):
        w = one_token(q[t], pg.keys(min(max(req[t], 0), 2), j), 64, 0.2, U[BF16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


def test_offsets_beyond_32_bits():
    """A cache of more than 2**32 elements, read at its far end."""
    rows, D = (1 << 32) // 512 + 4096, 512
    cache = torch.zeros(rows, D, dtype=BF16, device=DEV)
    g = gen(16)
    cache[-2048:] = torch.randn(2048, D, generator=g, device=DEV).to(BF16)
    q = torch.randn(2, 16, D, generator=g, device=DEV).to(BF16)
    pick = torch.randint(rows - 2048, rows, (2, 150), generator=g, device=DEV).int()
    o, lse = satk.latent_attend_rows(q, cache, pick, latent_dim=448, scale=0.05)
    table = i32([[rows // 16 - 3, rows // 16 - 1], [rows // 16 - 2, 0]])
    o2, _ = satk.latent_attend(q, cache, i32([0, 1]), table, i32([32, 16]), block_size=16,
                               stride_rows=16, latent_dim=448, scale=0.05)
    for t in range(2):
        w = one_token(q[t], cache[pick[t].long()], 448, 0.05, U[BF16])
        assert_close(o[t], w[0], w[2], f"rows, token {t}")
        first = int(table[t, 0]) * 16
        keys = cache[first:first + 16]
        if t == 0:
            keys = torch.cat([keys, cache[int(table[0, 1]) * 16:][:16]])
        w = one_token(q[t], keys, 448, 0.05, U[BF16])
        assert_close(o2[t], w[0], w[2], f"paged, token {t}")


# (dtype, heads, latent, tail, k, counts or None)
ROWS = [
    (BF16, 16, 128, 32, 64, [64, 0, 1, 63]), (BF16, 64, 512, 64, 200, [200, 129]),
    (F16, 20, 256, 64, 512, [512, 400, 65]), (BF16, 128, 384, 64, 130, None),
    (BF16, 100, 512, 32, 2048, [2048, 1365]), (F16, 1, 32, 0, 1, None),
    (BF16, 6, 30, 2, 77, [77, 12]), (BF16, 33, 448, 16, 96, [5])]


@pytest.mark.parametrize("case", range(len(ROWS)))
def test_rows(case):
    dtype, H, dl, dr, k, counts = ROWS[case]
    g, rng = gen(200 + case), np.random.RandomState(case)
    D, T, N = dl + dr, len(counts) if counts else 3, 4096
    cache = latent_rows(g, N, D, dtype)
    rows = np.full((T, k + 3), 12345678, dtype=np.int32)  # columns past k are not read
    for t in range(T):
        rows[t, :k] = rng.choice(N, k, replace=case % 2 == 0)
        rows[t, :k][rng.rand(k) < 0.1] = -1
        if counts:
            rows[t, counts[t]:k] = 10**8  # nor entries past the count
    named = set(rows[rows < N].tolist()) - {-1}
    cache[torch.tensor(sorted(set(range(N)) - named), device=DEV)] = float("nan")
    q = torch.randn(T, H, D, generator=g, device=DEV).to(dtype)
    scale = 1.3 / math.sqrt(D)
    out, check = guarded16((T, H, dl), dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = satk.latent_attend_rows(q, cache, i32(rows), k=k, latent_dim=dl, scale=scale,
                                     counts=i32(counts) if counts else None, out=out,
                                     status=status)
    torch.cuda.synchronize()
    check("latent_attend_rows")
    assert int(status.item()) == 0
    for t in range(T):
        at = rows[t, :counts[t] if counts else k]
        at = at[at >= 0].astype(np.int64)
        w = one_token(q[t], cache[torch.from_numpy(at).to(DEV)], dl, scale, U[dtype])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


def test_rows_bad_row_and_extreme_scores():
    """A row past the cache raises its bit and is skipped; scores of any size
    (a maximum that keeps growing along the keys, equal scores, -inf scores)
    give the definition's weights."""
    g = gen(17)
    dl, D, k = 128, 144, 320
    cache = latent_rows(g, 1000, D, BF16)
    cache[:, dl:] = 0
    cache[:, dl] = torch.arange(1000, device=DEV) * 0.5  # scores rise along the rows
    cache[5, dl + 1] = float("-inf")                     # a score of -inf
    q = torch.randn(3, 16, D, generator=g, device=DEV).to(BF16)
    q[:, :, dl:] = 0
    q[1, :, dl] = 3.0
    q[2, :, dl] = -2.0
    q[0, :, dl + 1] = 1.0
    rows = torch.arange(k, device=DEV).int().repeat(3, 1)
    rows[1:, 5] = 6  # row 5 only where its column counts
    rows[1, 7] = 1000
    rows[2, 7] = 2**31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = satk.latent_attend_rows(q, cache, rows, latent_dim=dl, scale=1.0, status=status)
    assert int(status.item()) == satk.STATUS_BAD_ROW
    for t in range(3):
        at = rows[t][rows[t] < 1000].long()
        if t == 0:
            at = at[at != 5]  # weight 0
        w = one_token(q[t], cache[at], dl, 1.0, U[BF16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("dl", [64, 128, 192, 256, 320, 384, 448, 512])
@pytest.mark.parametrize("dr,H,block", [(0, 16, 64), (64, 16, 16), (32, 33, 2), (48, 24, 8)])
def test_many_tiles_a_processor(dl, dr, H, block):
    """Enough keys that every SM goes through its stages several times, for
    every split of the columns, in pages that lie together and tiny ones, and
    the same rows as a selection."""
    g, rng = gen(dl + dr), np.random.RandomState(dl)
    D, R = dl + dr, 24
    ends = [int(x) for x in rng.randint(2500, 3500, R)]
    pg = Paged(g, rng, ends, D, block, BF16)
    q = torch.randn(R, H, D, generator=g, device=DEV).to(BF16)
    o, lse, st = run_paged(q, pg, range(R), ends, dl, 0.05)
    rows = np.full((R, max(ends)), -1, dtype=np.int32)
    for t in range(R):
        rows[t, :ends[t]] = rng.permutation(pg.rows(t, np.arange(ends[t])).numpy())
    o2, lse2 = satk.latent_attend_rows(q, pg.cache, i32(rows), latent_dim=dl, scale=0.05)
    assert st == 0
    for t in range(R):
        w = one_token(q[t], pg.keys(t, np.arange(ends[t])), dl, 0.05, U[BF16])
        assert_close(o[t], w[0], w[2], f"paged out, token {t}")
        assert_close(lse[t], w[1], w[3], f"paged lse, token {t}")
        assert_close(o2[t], w[0], w[2], f"rows out, token {t}")
        assert_close(lse2[t], w[1], w[3], f"rows lse, token {t}")


@pytest.mark.parametrize("H,new,context", [(16, 24, 3000), (64, 3, 2900), (6, 40, 1500)])
def test_many_tiles_of_trees(H, new, context):
    g, rng = gen(H), np.random.RandomState(H)
    dl, D, R, words = 256, 288, 8, 2
    lens = [int(c) + new for c in rng.randint(context - 500, context, R)]
    lens[3] = new  # nothing but drafted tokens
    pg = Paged(g, rng, lens, D, 16, F16)
    bits = np.concatenate([make_tree(rng, new, words) for _ in range(R)])
    req, ends = np.repeat(np.arange(R), new), np.repeat([n - new for n in lens], new)
    q = torch.randn(R * new, H, D, generator=g, device=DEV).to(F16)
    o, lse, st = run_paged(q, pg, req, ends, dl, 0.05, dtype=F16,
                           tree=torch.from_numpy(bits.view(np.int32)).to(DEV))
    assert st == 0
    for t in range(0, R * new, 5):
        j = list(range(ends[t])) + [ends[t] + b for b in range(64)
                                    if int(bits[t, b // 32]) >> (b % 32) & 1]
        w = one_token(q[t], pg.keys(req[t], j), dl, 0.05, U[F16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


def test_more_tokens_than_one_plan():
    """More tokens than one launch plans, most of them short."""
    g, rng = gen(5), np.random.RandomState(5)
    T, D, dl, N = 17000, 48, 32, 3000
    cache = latent_rows(g, N, D, BF16)
    rows = torch.randint(0, N, (T, 9), generator=g, device=DEV).int()
    counts = torch.randint(0, 10, (T,), generator=g, device=DEV).int()
    q = torch.randn(T, 3, D, generator=g, device=DEV).to(BF16)
    o, lse = satk.latent_attend_rows(q, cache, rows, counts=counts, latent_dim=dl, scale=0.1)
    for t in list(range(0, T, 997)) + [16383, 16384, T - 1]:
        n = int(counts[t])
        w = one_token(q[t], cache[rows[t, :n].long()], dl, 0.1, U[BF16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("scale", [-0.15, 0.0])
def test_scales_of_any_sign(scale):
    g, rng = gen(61), np.random.RandomState(61)
    pg = Paged(g, rng, [200, 65], 96, 16, BF16)
    q = torch.randn(2, 16, 96, generator=g, device=DEV).to(BF16)
    o, lse, _ = run_paged(q, pg, [0, 1], [200, 65], 64, scale)
    rows = torch.stack([pg.rows(0, np.arange(65)), pg.rows(1, np.arange(65))]).int().to(DEV)
    o2, lse2 = satk.latent_attend_rows(q, pg.cache, rows, latent_dim=64, scale=scale)
    for t, n in ((0, 200), (1, 65)):
        w = one_token(q[t], pg.keys(t, np.arange(n)), 64, scale, U[BF16])
        assert_close(o[t], w[0], w[2], f"paged out, token {t}")
        assert_close(lse[t], w[1], w[3], f"paged lse, token {t}")
        w = one_token(q[t], pg.keys(t, np.arange(65)), 64, scale, U[BF16])
        assert_close(o2[t], w[0], w[2], f"rows out, token {t}")
        assert_close(lse2[t], w[1], w[3], f"rows lse, token {t}")
    case = expanded_case(g, BF16, 2, 64, 32, 64, [40, 3], [0, 9])
    q, k, tail, v, ts, ks, ends = case
    o, lse = satk.latent_attend_expanded(q, k, tail, v, i32(ts), i32(ks), i32(ends), scale=scale)
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, scale)


@pytest.mark.parametrize("block", [64, 16, 8, 4])
def test_page_cut_by_the_cache_end(block):
    """A block whose last rows lie past the cache: they are not seen, the bit
    is raised, and what a box brings in their place does not matter."""
    g = gen(63)
    rows = 4 * block - 3
    cache = latent_rows(g, rows, 96, F16)
    table, ends = i32([[1, 3], [0, 2]]), [2 * block, 2 * block - 1]
    q = torch.randn(2, 16, 96, generator=g, device=DEV).to(F16)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = satk.latent_attend(q, cache, i32([0, 1]), table, i32(ends), block_size=block,
                                stride_rows=block, latent_dim=64, scale=0.2, status=status)
    assert int(status.item()) == satk.STATUS_BAD_ROW
    for t, at in ((0, list(range(block, 2 * block)) + list(range(3 * block, rows))),
                  (1, list(range(block)) + list(range(2 * block, 3 * block - 1)))):
        w = one_token(q[t], cache[torch.tensor(at, device=DEV)], 64, 0.2, U[F16])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("selected", [False, True])
def test_nan_next_to_what_is_seen(selected):
    """Rows between a request's keys and its block's end, row 0 of the cache
    (what stands in for skipped entries) and other requests' rows are NaN, in
    every tile of a long context; heads of one token see one NaN query alone."""
    g, rng = gen(65), np.random.RandomState(65)
    ends = [1000, 7, 0, 64, 129]
    pg = Paged(g, rng, ends, 160, 64, BF16)
    q = torch.randn(5, 24, 160, generator=g, device=DEV).to(BF16)
    q[0, 3, 5] = float("nan")
    if selected:
        rows = np.full((5, 1100), -1, dtype=np.int32)
        for t, n in enumerate(ends):
            rows[t, np.sort(rng.permutation(1100)[:n])] = pg.rows(t, np.arange(n)).numpy()
        free = sorted(set(range(pg.cache.shape[0])) - set(rows.ravel().tolist()))
        pg.cache[torch.tensor(free, device=DEV)] = float("inf")
        o, lse = satk.latent_attend_rows(q, pg.cache, i32(rows), latent_dim=128, scale=0.1)
    else:
        o, lse, _ = run_paged(q, pg, range(5), ends, 128, 0.1)
    assert torch.isnan(o[0, 3]).all() and torch.isnan(lse[0, 3])
    for t in range(5):
        heads = [h for h in range(24) if (t, h) != (0, 3)]
        w = one_token(q[t, heads], pg.keys(t, np.arange(ends[t])), 128, 0.1, U[BF16])
        assert_close(o[t, heads], w[0], w[2], f"out, token {t}")
        assert_close(lse[t, heads], w[1], w[3], f"lse, token {t}")


def test_step_tables_without_requests():
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    t = satk.step_tables(e, e, i32([1, 2]), torch.zeros(0, 4, dtype=torch.int32, device=DEV),
                         tokens=3, block_size=16, stride_rows=16)
    assert t.token_starts.tolist() == [0] and t.blocks_used.tolist() == [0]
    assert t.slots.tolist() == [-1] * 3 and t.row_ends.tolist() == [0] * 3


def test_attend_empty_calls():
    cache = torch.zeros(0, 96, dtype=BF16, device=DEV)
    q = torch.randn(2, 4, 96, device=DEV).to(BF16)
    o, lse = satk.latent_attend_rows(q, cache, i32([[-1], [-1]]), latent_dim=64, scale=1.0)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    o, lse = satk.latent_attend(q, cache, i32([0, 0]), torch.zeros(1, 0, dtype=torch.int32, device=DEV),
                                i32([5, 0]), block_size=16, stride_rows=16, latent_dim=64,
                                scale=1.0)
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
    o, lse = satk.latent_attend_rows(q[:0], cache, torch.zeros(0, 3, dtype=torch.int32, device=DEV),
                                     latent_dim=64, scale=1.0)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


# --- expanded ---------------------------------------------------------------

# (dtype, heads, nope, tail, value, new tokens, context)
EXPANDED = [
    (BF16, 2, 64, 32, 64, [130, 1, 64], [0, 0, 0]), (F16, 3, 128, 64, 128, [257], [100]),
    (BF16, 1, 128, 0, 96, [5, 300], [700, 3]), (BF16, 2, 32, 16, 32, [128, 128, 129], [0, 1, 64]),
    (BF16, 4, 112, 48, 48, [40], [0]), (F16, 2, 20, 6, 10, [33, 9], [0, 40]),
    (BF16, 2, 192, 64, 128, [150], [31])]


def expanded_case(g, dtype, H, dn, dr, dv, new, context):
    T, lens = sum(new), [n + c for n, c in zip(new, context)]
    S = sum(lens)
    q = torch.randn(T, H, dn + dr, generator=g, device=DEV).to(dtype)
    k = torch.randn(S, H, dn, generator=g, device=DEV).to(dtype)
    tail = torch.randn(S, dr, generator=g, device=DEV).to(dtype) if dr else None
    v = (torch.randn(S, H, dv, generator=g, device=DEV) + 0.5).to(dtype)
    ts, ks = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(lens)])
    ends = np.concatenate([c + 1 + np.arange(n) for c, n in zip(context, new)])
    return q, k, tail, v, ts, ks, ends


def expanded_check(q, k, tail, v, ts, ks, ends, o, lse, scale, skip=lambda t: False):
    u = U[q.dtype]
    full = k if tail is None else torch.cat([k, tail[:, None].expand(-1, k.shape[1], -1)], 2)
    for r in range(len(ts) - 1):
        for t in range(ts[r], ts[r + 1]):
            if skip(t):
                continue
            n = min(max(int(ends[t]), 0), int(ks[r + 1] - ks[r]))
            if n == 0:
                assert torch.all(o[t] == 0) and torch.all(torch.isneginf(lse[t]))
                continue
            at = slice(int(ks[r]), int(ks[r]) + n)
            w = attention64(q[t].double(), full[at].transpose(0, 1).double(),
                            v[at].transpose(0, 1).double(), scale, u)
            assert_close(o[t], w[0], w[2], f"out, token {t}")
            assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("case", range(len(EXPANDED)))
def test_expanded(case):
    dtype, H, dn, dr, dv, new, context = EXPANDED[case]
    q, k, tail, v, ts, ks, ends = expanded_case(gen(300 + case), *EXPANDED[case])
    scale = 1.3 / math.sqrt(dn + dr)
    out, check = guarded16((q.shape[0], H, dv), dtype)
    o, lse = satk.latent_attend_expanded(q, k, tail, v, i32(ts), i32(ks), i32(ends), scale=scale,
                                         out=out)
    torch.cuda.synchronize()
    check("latent_attend_expanded")
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_expanded_masks(dtype):
    """Ends of any kind: zero, past the request, not ascending; NaN and
    infinity in keys and values that no token or only some tokens see."""
    g = gen(31)
    q, k, tail, v, ts, ks, _ = expanded_case(g, dtype, 2, 64, 32, 64, [140, 60], [60, 0])
    ends = np.random.RandomState(3).randint(0, 150, 200)
    ends[:3], ends[5], ends[150:] = 0, 190, np.arange(50) + 1
    k[195:200], v[195:200] = float("nan"), float("inf")   # seen by no token
    v[170, :, 3] = float("nan")                           # seen by token 5 alone
    k[250, :, 1] = float("inf")                           # request 1's key 50: not seen
    ends[140:] = np.minimum(ends[140:], 50)
    o, lse = satk.latent_attend_expanded(q, k, tail, v, i32(ts), i32(ks), i32(ends), scale=0.2)
    assert not torch.isfinite(o[5]).all()
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, 0.2, skip=lambda t: t == 5)


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_expanded_layouts(pad):
    """Strides of their own (16-byte aligned and not), key and value halves of
    one projection's output, heads before tokens, tokens outside every request."""
    g = gen(33)
    T, S, H, dn, dr, dv = 150, 180, 3, 64, 16, 32
    q = torch.randn(H, T, dn + dr + pad, generator=g, device=DEV).to(BF16).transpose(0, 1)[..., :dn + dr]
    kv = torch.randn(S, H, dn + dv + pad, generator=g, device=DEV).to(BF16)
    k, v = kv[..., :dn], kv[..., dn:dn + dv]
    tail = torch.randn(S, dr + pad, generator=g, device=DEV).to(BF16)[:, :dr]
    ts, ks = np.array([4, 4, 140]), np.array([0, 20, 170])
    ends = np.full(T, 10**6)
    canvas = torch.full((T, H, dv + 5), -7.0, dtype=BF16, device=DEV)
    o, lse = satk.latent_attend_expanded(q, k, tail, v, i32(ts), i32(ks), i32(ends), scale=0.2,
                                         out=canvas[..., :dv])
    assert torch.all(canvas[..., dv:] == -7.0)
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, 0.2)
    outside = torch.tensor([t for t in range(T) if t < 4 or t >= 140], device=DEV)
    assert torch.all(o[outside] == 0) and torch.all(torch.isneginf(lse[outside]))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dv", [64, 128])
def test_expanded_with_garbage_left_in_shared_memory(dtype, dv):
    """Last tiles of few tokens over several key tiles, right after a kernel
    that fills shared memory with NaN: nothing is read before it has arrived."""
    g = gen(36)
    new, context = [300, 260, 40, 1], [0, 100, 600, 900]
    q, k, tail, v, ts, ks, ends = expanded_case(g, dtype, 4, 64, 32, dv, new, context)
    nan = torch.full((4096, 544), float("nan"), dtype=dtype, device=DEV)
    fill = torch.randint(0, 4096, (256, 512), generator=g, device=DEV).int()
    fq = torch.zeros(256, 64, 544, dtype=dtype, device=DEV)
    args = (q, k, tail, v, i32(ts), i32(ks), i32(ends))
    for _ in range(4):
        satk.latent_attend_rows(fq, nan, fill, latent_dim=512, scale=1.0)
        o, lse = satk.latent_attend_expanded(*args, scale=0.2)
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, 0.2)


def test_expanded_long_keys_and_few_tokens():
    """One sub-tile or one token over more key tiles than the panels' ring and
    its barriers hold, next to two full sub-tiles that end apart."""
    g = gen(37)
    for dn, dr, dv in ((32, 16, 32), (64, 0, 64), (128, 64, 128), (192, 64, 96)):
        new, context = [3, 1, 256, 129], [4000, 2500, 1500, 3000]
        q, k, tail, v, ts, ks, ends = expanded_case(g, BF16, 2, dn, dr, dv, new, context)
        ends[4:132] = np.minimum(ends[4:132], 100)  # the first sub-tile ends early
        o, lse = satk.latent_attend_expanded(q, k, tail, v, i32(ts), i32(ks), i32(ends), scale=0.1)
        expanded_check(q, k, tail, v, ts, ks, ends, o, lse, 0.1, skip=lambda t: t % 9 > 1)


def test_expanded_many_requests_and_graph():
    g = gen(35)
    new = [1 + (i * 7) % 23 for i in range(150)]
    q, k, tail, v, ts, ks, ends = expanded_case(g, BF16, 2, 32, 16, 32, new, [0] * 150)
    args = (q, k, tail, v, i32(ts), i32(ks), i32(ends))
    o, lse = satk.latent_attend_expanded(*args, scale=0.2)
    expanded_check(q, k, tail, v, ts, ks, ends, o, lse, 0.2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = satk.latent_attend_expanded(*args, scale=0.2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, l2)


# --- merge, store, tables ---------------------------------------------------

@pytest.mark.parametrize("dtype,W,T,H,dv,pad", [
    (BF16, 2, 3, 5, 64, 0), (F16, 8, 17, 16, 512, 0), (BF16, 3, 4, 2, 30, 0), (F16, 5, 2, 3, 32, 3),
    (BF16, 1, 1, 1, 8, 0), (BF16, 64, 2, 2, 48, 8)])
def test_merge(dtype, W, T, H, dv, pad):
    g = gen(41)
    parts = torch.randn(W, T, H, dv + pad, generator=g, device=DEV).to(dtype)[..., :dv]
    lse = torch.randn(W, T, H, generator=g, device=DEV) * 20
    dead = torch.rand(W, T, H, generator=g, device=DEV) < 0.3
    dead[:, 0, 0] = True
    lse[dead] = -math.inf
    parts[dead] = float("nan")  # what an empty part holds is not read
    out, check = guarded16((T, H, dv), dtype)
    o, l = satk.latent_merge(parts, lse, out=out)
    torch.cuda.synchronize()
    check("latent_merge")
    x = torch.where(dead[..., None], 0.0, parts.double())
    total = torch.logsumexp(lse.double(), 0)
    w = torch.where(dead, 0.0, torch.exp(lse.double() - torch.where(total == -math.inf, 0.0, total)))
    want, mass = (x * w[..., None]).sum(0), (x.abs() * w[..., None]).sum(0)
    # exponents of up to 100 in 32 bits: 100 2^-23 each
    assert_close(o, want, U[dtype] * want.abs() + 3e-5 * mass + 2.0**-25, "out")
    assert_close(l, total, 1e-5 + 1e-6 * total.abs(), "lse")


def test_merge_joins_attention_over_split_keys():
    g = gen(43)
    cache = latent_rows(g, 600, 160, BF16)
    q = torch.randn(4, 16, 160, generator=g, device=DEV).to(BF16)
    rows = torch.arange(600, device=DEV).int().repeat(4, 1)
    parts = [satk.latent_attend_rows(q, cache, rows[:, w::3].contiguous(), latent_dim=128, scale=0.1)
             for w in range(3)]
    o, lse = satk.latent_merge(torch.stack([p[0] for p in parts]),
                               torch.stack([p[1] for p in parts]))
    for t in range(4):
        w = one_token(q[t], cache, 128, 0.1, U[BF16])
        mass = w[2]
        # the parts' own rounding on top: the tolerance of each part again
        assert_close(o[t], w[0], 2 * mass + U[BF16] * 2, "out")
        assert_close(lse[t], w[1], 2 * w[3], "lse")


@pytest.mark.parametrize("dtype,T,dl,dr,interleaved,norm,rotate,ld,pad", [
    (BF16, 9, 512, 64, False, True, True, 576, 0), (F16, 33, 384, 32, True, True, True, 416, 0),
    (BF16, 5, 100, 6, True, True, True, 131, 1), (BF16, 4, 128, 0, False, True, False, 128, 8),
    (F16, 3, 64, 64, False, False, True, 200, 0), (BF16, 2, 7, 2, False, False, False, 9, 0),
    (BF16, 1, 512, 64, True, True, True, 576, 3)])
def test_store(dtype, T, dl, dr, interleaved, norm, rotate, ld, pad):
    g = gen(51)
    rows, n_pos = 40, 500
    x = (3 * torch.randn(T, dl + pad, generator=g, device=DEV)).to(dtype)[:, :dl]
    tail = torch.randn(T, dr + pad, generator=g, device=DEV).to(dtype)[:, :dr] if dr else None
    weight = torch.rand(dl, generator=g, device=DEV) + 0.5 if norm else None
    angle = torch.rand(n_pos, max(dr // 2, 1), generator=g, device=DEV) * 6.28
    cs = torch.cat([angle.cos(), angle.sin()], 1) if rotate else None
    pos = i32(np.random.RandomState(5).randint(0, n_pos, T))
    slots = np.random.RandomState(6).permutation(rows)[:T]
    if T > 3:
        slots[1] = -1
    buf, check = guarded16((rows, ld), dtype)
    buf.fill_(7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = satk.latent_store(x, tail, i32(slots), buf, weight=weight, eps=1e-5, cos_sin=cs,
                            positions=pos if rotate else None, interleaved=interleaved,
                            status=status)
    torch.cuda.synchronize()
    check("latent_store")
    assert int(status.item()) == 0
    want = torch.full((rows, ld), 7.0, dtype=torch.float64, device=DEV)
    y = x.double()
    if norm:
        y = y / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-5) * weight.double()
    if dr:
        z = tail.double()
        if rotate:
            c, s = cs.double()[pos.long()].chunk(2, 1)
            a, b = (z[:, 0::2], z[:, 1::2]) if interleaved else z.chunk(2, 1)
            r0, r1 = a * c - b * s, a * s + b * c
            z = torch.stack([r0, r1], 2).flatten(1) if interleaved else torch.cat([r0, r1], 1)
        y = torch.cat([y, z], 1)
    for t in range(T):
        if slots[t] >= 0:
            want[slots[t], :dl + dr] = y[t]
    # one rounding, and fp32 arithmetic on values up to about 20
    assert_close(got, want, U[dtype] * want.abs() + 2e-5, "cache")
    if not norm and not rotate:
        assert torch.equal(got.double(), want)


def test_store_bad_slots_and_positions():
    x = torch.ones(4, 64, dtype=BF16, device=DEV)
    tail = torch.ones(4, 16, dtype=BF16, device=DEV)
    cs = torch.ones(10, 16, device=DEV)
    for slots, pos, bit in (([0, 99, 2, -5], [0, 0, 0, 99], satk.STATUS_BAD_ROW),
                            ([0, 1, 2, 3], [0, -1, 9, 10], satk.STATUS_BAD_POSITION)):
        cache = torch.full((8, 80), 7.0, dtype=BF16, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        satk.latent_store(x, tail, i32(slots), cache, cos_sin=cs, positions=i32(pos), status=st)
        assert int(st.item()) == bit
        kept = [s for s, p in zip(slots, pos) if 0 <= s < 8 and 0 <= p < 10]
        for r in range(8):
            assert torch.all(cache[r, :64] == (1.0 if r in kept else 7.0))


def tables_oracle(ctx, new, free, table, T, B, stride, W, rank, drafted):
    """Request by request, token by token."""
    local = lambda p: sum(1 for _ in range(rank, p, W))  # noqa: E731
    table, status, used, width = table.copy(), 0, 0, table.shape[1]
    starts, lens = [0], []
    req, pos, ends, slots = ([] for _ in range(4))
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        have, need = (min(-(-local(x) // B), width) for x in (c, c + n))
        here = {b: int(table[r, b]) for b in range(have)}
        for b in range(have, need):
            if used < len(free):
                table[r, b] = here[b] = int(free[used])
            used += 1
        for p in range(c, c + n):
            if len(req) >= T:
                status |= satk.STATUS_TOO_MANY_TOKENS
                break
            slot = -1
            if p % W == rank:
                l = p // W
                block = here.get(l // B, -1)
                if block < 0:
                    status |= satk.STATUS_NO_BLOCK
                else:
                    slot = block * stride + l % B
            req.append(r), pos.append(p), slots.append(slot)
            ends.append(local(c) if drafted else local(p + 1))
        starts.append(min(T, starts[-1] + n))
        lens.append(local(c + n))
    pad = T - len(req)
    return (table, starts, lens, req + [0] * pad, pos + [0] * pad, ends + [0] * pad,
            slots + [-1] * pad, [min(used, len(free))], status)


@pytest.mark.parametrize("R,new_max,ctx_max,B,W,rank,drafted,T,n_free,width", [
    (5, 1, 100, 16, 1, 0, False, 5, 50, 9), (5, 9, 100, 16, 4, 2, False, 40, 50, 4),
    (1, 1, 1, 1, 1, 0, False, 1, 1, 3), (40, 30, 300, 7, 3, 0, True, 2000, 900, 20),
    (33, 20, 60, 8, 2, 1, False, 100, 30, 4), (3, 5, 40, 16, 1, 0, False, 20, 0, 1),
    (700, 6, 20, 4, 1, 0, False, 4000, 5000, 8), (4, 3, 5, 4, 8, 7, False, 0, 8, 3)])
def test_step_tables(R, new_max, ctx_max, B, W, rank, drafted, T, n_free, width):
    rng = np.random.RandomState(R)
    ctx, new = rng.randint(0, ctx_max, R), rng.randint(0, new_max + 1, R)
    if R > 30:
        ctx[3], new[4] = -5, -1  # count as 0
    blocks = rng.permutation(n_free + R * width)
    free, table = blocks[:n_free].astype(np.int32), blocks[n_free:].reshape(R, width).astype(np.int32)
    stride = B + 1
    want = tables_oracle(ctx, new, free, table, T, B, stride, W, rank, drafted)
    dt = i32(table)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    sizes = (R + 1, R, T, T, T, T, 1)
    bufs, checks = zip(*(guarded((n,)) for n in sizes))
    got = satk.step_tables(i32(ctx), i32(new), i32(free), dt, tokens=T, block_size=B,
                           stride_rows=stride, W=W, dcp_rank=rank, drafted=drafted,
                           out=satk.StepTables(*bufs), status=st)
    torch.cuda.synchronize()
    for c in checks:
        c("step_tables")
    assert np.array_equal(dt.cpu().numpy(), want[0]), "block table"
    for name, x, y in zip(satk.StepTables._fields, got, want[1:8]):
        assert x.cpu().tolist() == list(y), name
    assert int(st.item()) == want[8]
    plain = satk.step_tables(i32(ctx), i32(new), i32(free), i32(table), tokens=T, block_size=B,
                             stride_rows=stride, W=W, dcp_rank=rank, drafted=drafted)
    for x, y in zip(plain, got):
        assert torch.equal(x, y)


def test_binding_refusals():
    x = torch.zeros(4, 8, 32, dtype=BF16, device=DEV)
    c = torch.zeros(16, 32, dtype=BF16, device=DEV)
    r = torch.zeros(4, 4, dtype=torch.int32, device=DEV)
    kw = dict(latent_dim=16, scale=1.0)
    for bad in (lambda: satk.latent_attend_rows(x.float(), c, r, **kw),
                lambda: satk.latent_attend_rows(x, c.half(), r, **kw),
                lambda: satk.latent_attend_rows(x, c[:, :16], r, **kw),
                lambda: satk.latent_attend_rows(x, c, r.long(), **kw),
                lambda: satk.latent_attend_rows(x, c, r[:3], **kw),
                lambda: satk.latent_attend_rows(x, c, r, latent_dim=33, scale=1.0),
                lambda: satk.latent_attend_rows(x, c, r, latent_dim=16, scale=float("nan")),
                lambda: satk.latent_attend_rows(x, c, r, out=x, **kw),
                lambda: satk.latent_attend_rows(x, c, r, workspace=torch.zeros(1, device=DEV), **kw),
                lambda: satk.latent_attend_rows(x.transpose(1, 2), c, r, **kw),
                lambda: satk.latent_merge(x[None], torch.zeros(1, 4, 7, device=DEV)),
                lambda: satk.latent_store(c[:4], None, r[0], c, weight=torch.zeros(31, device=DEV)),
                lambda: satk.latent_attend_expanded(x, x, c[:3], x, r[0], r[0], r[0], scale=1.0),
                lambda: satk.step_tables(r[0], r[0], r[0], r.float(), tokens=4, block_size=4,
                                         stride_rows=4)):
        with pytest.raises(satk.SatkError):
            bad()
