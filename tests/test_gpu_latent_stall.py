"""What comes out of the attention over cache rows when a wait inside the GPU
is given up.  No wait is made to run out: the debug build, asked to, takes the
last result of every CTA for one after a given-up wait, once all of the CTA's
copies and products are done."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from sparse_attention_indexer_radix_gb300 import build as satk_build
from test_gpu_latent import BF16, DEV, Paged, U, assert_close, gen, i32, one_token

pytestmark = pytest.mark.gpu
STALL, FIRST_CLEAR = 256, 1


@pytest.fixture(scope="module")
def dbg():
    return binding.load(satk_build.build(debug=True))


@pytest.mark.parametrize("selected", [False, True])
@pytest.mark.parametrize("lens", [[5000, 3000], [40] * 400, [900] * 170 + [0, 64]])
def test_a_given_up_wait_shows_in_the_results(dbg, selected, lens):
    """Results of requests that are cut over CTAs, whole, and several to a CTA:
    each is right or NaN throughout, its lse with it, whether the caller passes a
    status word or not; and right again once nothing is asked for."""
    g, rng = gen(71), np.random.RandomState(71)
    R, H, dl, D = len(lens), 16, 64, 96
    pg = Paged(g, rng, lens, D, 16, BF16)
    q = torch.randn(R, H, D, generator=g, device=DEV).to(BF16)
    if selected:
        rows = np.full((R, max(lens)), -1, dtype=np.int32)
        for t, n in enumerate(lens):
            rows[t, :n] = pg.rows(t, np.arange(n)).numpy()
        rows = i32(rows)
        call = lambda **kw: satk.latent_attend_rows(q, pg.cache, rows, latent_dim=dl,  # noqa: E731
                                                    scale=0.1, **kw)
    else:
        args = (q, pg.cache, i32(range(R)), i32(pg.table), i32(lens))
        call = lambda **kw: satk.latent_attend(*args, block_size=16, stride_rows=16,  # noqa: E731
                                               latent_dim=dl, scale=0.1, **kw)
    with binding.routed_to(dbg):
        dbg.satk_debug_flags(FIRST_CLEAR)
        status = i32([0])
        good = call(status=status)
        assert int(status.item()) == 0
        dbg.satk_debug_flags(2)
        try:
            bad = call(status=status)
            silent = call()
            torch.cuda.synchronize()
        finally:
            assert dbg.satk_debug_flags(FIRST_CLEAR) == STALL
        again = call()
    for t in range(0, R, max(1, R // 20)):
        w = one_token(q[t], pg.keys(t, np.arange(lens[t])), dl, 0.1, U[BF16])
        assert_close(good[0][t], w[0], w[2], f"out, token {t}")
        assert_close(good[1][t], w[1], w[3], f"lse, token {t}")
    assert int(status.item()) == satk.STATUS_STALLED
    for o, lse in (bad, silent):
        lost = torch.isnan(o).all(2)
        assert lost.any() and torch.equal(lost, torch.isnan(lse))
        assert torch.equal(o[~lost], good[0][~lost]) and torch.equal(lse[~lost], good[1][~lost])
        if R == 2:
            assert lost.all()  # every CTA holds a part of one of the two
    for a, b in zip(good, again):
        assert torch.equal(a, b)


def test_the_normal_build_takes_no_notice():
    from sparse_attention_indexer_radix_gb300 import build
    build.build()
    assert binding.lib().satk_debug_flags(2) == 0
    g = gen(72)
    cache = torch.randn(64, 96, generator=g, device=DEV).to(BF16)
    q = torch.randn(1, 4, 96, generator=g, device=DEV).to(BF16)
    o, lse = satk.latent_attend_rows(q, cache, i32([list(range(64))]), latent_dim=64,
                                     scale=1 / math.sqrt(96))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
