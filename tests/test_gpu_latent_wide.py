"""Masks at the widest rows (512 values and a tail, 64 score columns: two stages
in two halves), and the latent-cache operators without attention on side streams
and in graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from test_gpu_latent import (BF16, DEV, F16, U, Paged, assert_close, gen, i32, make_tree,
                             one_token, run_paged)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


# (dtype, heads, latent, tail, block): pages in boxes and by copies; groups of 4,
# 3, 64, 1 and 2 tokens, two head chunks; one to eight blocks of values
WIDE = [(BF16, 16, 512, 64, 64), (F16, 16, 512, 64, 12), (BF16, 21, 512, 32, 16),
        (BF16, 21, 512, 64, 12), (F16, 1, 512, 64, 128), (BF16, 64, 512, 0, 32),
        (BF16, 64, 512, 64, 12), (BF16, 128, 512, 64, 64), (F16, 128, 512, 64, 4),
        (BF16, 32, 448, 64, 16), (BF16, 32, 448, 16, 12)]


def not_finite_where_it_counts(o, q, keys, row):
    """A token's output [H, dl] where it sees a row that is not finite: NaN or
    infinity for every head whose score of it is not finite, but for -inf, whose
    weight is 0."""
    score = (q.double() @ keys[row].double())
    heads = torch.isnan(score) | torch.isposinf(score)
    assert not torch.isfinite(score).any()
    assert not torch.isfinite(o[heads]).all(1).any()


@pytest.mark.parametrize("odd", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_chunks_of_wide_rows(case, odd):
    """Causal tokens that see different keys of a tile; the last one's row is not
    finite, so it has to be kept from the others in its group."""
    dtype, H, dl, dr, block = WIDE[case]
    g, rng = gen(91 + case), np.random.RandomState(case)
    new, context = [9, 1, 70], [600, 64, 0]
    lens = [a + b for a, b in zip(new, context)]
    pg = Paged(g, rng, lens, dl + dr, block, dtype)
    for r, n in enumerate(lens):
        pg.cache[pg.rows(r, [n - 1]).to(DEV), 3] = odd
    req = np.repeat(np.arange(len(new)), new)
    ends = np.concatenate([c + 1 + np.arange(n) for c, n in zip(context, new)])
    q = torch.randn(len(req), H, dl + dr, generator=g, device=DEV).to(dtype)
    o, lse, st = run_paged(q, pg, req, ends, dl, 0.05, dtype=dtype)
    assert st == 0
    for t, r in enumerate(req):
        if ends[t] == lens[r]:
            not_finite_where_it_counts(o[t], q[t], pg.keys(r, np.arange(ends[t])), -1)
            continue
        w = one_token(q[t], pg.keys(r, np.arange(ends[t])), dl, 0.05, U[dtype])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


@pytest.mark.parametrize("case", range(len(WIDE)))
def test_trees_of_wide_rows(case):
    """Drafted trees behind contexts that end inside a tile; the rows of tokens
    without descendants are not finite and seen by themselves alone."""
    dtype, H, dl, dr, block = WIDE[case]
    g, rng = gen(191 + case), np.random.RandomState(case)
    new, context = [40, 7, 33], [500, 0, 63]
    lens = [a + b for a, b in zip(new, context)]
    pg = Paged(g, rng, lens, dl + dr, block, dtype)
    bits = np.concatenate([make_tree(rng, n, 2) for n in new])
    req, ends = np.repeat(np.arange(len(new)), new), np.repeat(context, new)
    path = [[b for b in range(64) if int(bits[t, b // 32]) >> (b % 32) & 1]
            for t in range(len(req))]
    first = np.cumsum([0] + new)
    leaf = np.zeros(len(req), dtype=bool)
    for t, r in enumerate(req):
        i = t - first[r]
        leaf[t] = not any(i in path[u] for u in range(first[r], first[r + 1]) if u != t)
        if leaf[t]:
            pg.cache[pg.rows(r, [context[r] + i]).to(DEV), 5] = float("inf" if t % 2 else "nan")
    assert leaf.any() and not leaf.all()
    q = torch.randn(len(req), H, dl + dr, generator=g, device=DEV).to(dtype)
    o, lse, st = run_paged(q, pg, req, ends, dl, 0.05, dtype=dtype,
                           tree=torch.from_numpy(bits.view(np.int32)).to(DEV))
    assert st == 0
    for t, r in enumerate(req):
        if leaf[t]:
            not_finite_where_it_counts(o[t], q[t], pg.keys(r, [context[r] + t - first[r]]), 0)
            continue
        j = list(range(ends[t])) + [ends[t] + b for b in path[t]]
        w = one_token(q[t], pg.keys(r, j), dl, 0.05, U[dtype])
        assert_close(o[t], w[0], w[2], f"out, token {t}")
        assert_close(lse[t], w[1], w[3], f"lse, token {t}")


def step(seed):
    """One step's tables and cache write, and a join, on buffers of their own:
    the calls, and what they write."""
    g, rng = gen(seed), np.random.RandomState(seed)
    R, T = 40, 200
    ctx, new = i32(rng.randint(0, 90, R)), i32(rng.randint(0, 6, R))
    free = i32(rng.permutation(400))
    table0 = i32(rng.permutation(R * 8).reshape(R, 8) + 400)
    table = table0.clone()
    out = satk.StepTables(*(i32(np.zeros(n)) for n in (R + 1, R, T, T, T, T, 1)))
    latent = torch.randn(T, 256, generator=g, device=DEV).to(BF16)
    tail = torch.randn(T, 32, generator=g, device=DEV).to(BF16)
    weight = torch.rand(256, generator=g, device=DEV)
    cos_sin = torch.rand(200, 32, generator=g, device=DEV)
    cache = torch.zeros((400 + R * 8) * 16, 288, dtype=BF16, device=DEV)
    parts = torch.randn(3, 20, 4, 64, generator=g, device=DEV).to(BF16)
    lse = torch.randn(3, 20, 4, generator=g, device=DEV)
    joined = torch.zeros(20, 4, 64, dtype=BF16, device=DEV)
    joined_lse = torch.zeros(20, 4, device=DEV)

    def run():
        table.copy_(table0)
        satk.step_tables(ctx, new, free, table, tokens=T, block_size=16, stride_rows=16, out=out)
        satk.latent_store(latent, tail, out.slots, cache, weight=weight, cos_sin=cos_sin,
                          positions=out.positions)
        satk.latent_merge(parts, lse, out=joined, lse_out=joined_lse)
    inputs = [ctx, new, latent, tail, parts, lse]
    return run, inputs, [table, *out, cache, joined, joined_lse]


def test_step_on_a_side_stream():
    run, _, results = step(5)
    run()
    torch.cuda.synchronize()
    want = [x.clone() for x in results]
    for x in results:
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    for a, b in zip(want, results):
        assert torch.equal(a, b)


def test_step_in_a_graph():
    """Captured once, replayed on other lengths, latents and parts."""
    run, inputs, results = step(5)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    eager, eager_inputs, want = step(5)
    for a, b, c in zip(inputs, eager_inputs, step(6)[1]):
        a.copy_(c)
        b.copy_(c)
    for x in results:
        x.zero_()
    graph.replay()
    eager()
    torch.cuda.synchronize()
    for a, b in zip(want, results):
        assert torch.equal(a, b)
