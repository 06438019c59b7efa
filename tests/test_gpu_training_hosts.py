"""Host-side conditions of the training calls on the GPU: first calls of threads,
threads that call at once, whole chains in one graph, the debug build."""
from __future__ import annotations

import threading

import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from sparse_attention_indexer_radix_gb300 import build as satk_build
from test_gpu_expanded_grad import Case
from test_gpu_latent import BF16, DEV, gen, i32, latent_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    satk_build.build()


def losses(seed):
    g = gen(seed)
    logits = torch.randn(6, 9001, generator=g, device=DEV).to(BF16)
    ids = torch.rand(6, 9001, generator=g, device=DEV).topk(200, dim=1).indices.int()
    x = torch.rand(6, 200, generator=g, device=DEV)
    one = torch.ones(1, device=DEV)

    def call():
        loss, lse = satk.distill_loss(logits, ids, x, kind="weights")
        return loss, lse, satk.distill_grad(logits, ids, x, lse, one, kind="weights")
    return call


def weights(seed, heads=48, D=320):
    g = gen(seed)
    cache = latent_rows(g, 700, D, BF16)
    q = torch.randn(5, heads, D, generator=g, device=DEV).to(BF16)
    rows = torch.randint(0, 700, (5, 333), generator=g, device=DEV).int()
    lse = torch.randn(5, heads, generator=g, device=DEV) + 20
    return lambda: (satk.latent_rows_weights(q, cache, rows, lse, scale=0.05),)


def gradients(seed, widths=(128, 64, 128)):
    c = Case(gen(seed), BF16, 2, *widths, [150, 70], [30, 0])
    c.forward()
    return lambda: tuple(x for x in c.grad() if x is not None)


CALLS = [(losses, (1,)), (weights, (2,)), (weights, (3, 128, 576)), (weights, (4, 5, 33)),
         (gradients, (5,)), (gradients, (6, (33, 3, 20)))]


@pytest.mark.parametrize("make,args", CALLS)
def test_first_call_of_a_thread(make, args):
    call = make(*args)
    want = tuple(x.clone() for x in call())
    torch.cuda.synchronize()
    got, errors = [], []

    def work():
        try:
            got.extend(call())
        except satk.SatkError as e:
            errors.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors and len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_threads_that_call_at_once():
    calls = [make(*args) for make, args in CALLS]
    want = [tuple(x.clone() for x in call()) for call in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(call, result):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = call()
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, result)):
                    wrong.append(call)
    threads = [threading.Thread(target=work, args=x) for x in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("make,args", CALLS)
def test_debug_build(make, args):
    call = make(*args)
    want = tuple(x.clone() for x in call())
    dbg = binding.load(satk_build.build(debug=True))
    with binding.routed_to(dbg):
        dbg.satk_debug_flags(1)
        got = call()
        assert dbg.satk_debug_flags(1) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_sparse_step_in_one_graph():
    """Selection, attention, weights, loss and gradient captured together and
    replayed on other scores."""
    g = gen(7)
    T, H, D, dl, k, S = 9, 16, 160, 128, 64, 500
    cache = latent_rows(g, S, D, BF16)
    q = torch.randn(T, H, D, generator=g, device=DEV).to(BF16)
    scores = torch.randn(T, S, generator=g, device=DEV)
    ends = i32([S, 3, 0, 64, 65, 400, 1, 200, 63])
    one = torch.ones(1, device=DEV)
    status = i32([0])

    def step():
        ids = satk.topk_rows(scores, k, row_ends=ends)
        # (the cache's rows are the tokens: one request in one block)
        rows, count = satk.dcp_emit_rows(ids, 1, 0, i32([0] * T) if first else req, table, S, S,
                                         status=status)
        out, lse = satk.latent_attend_rows(q, cache, rows, counts=count, latent_dim=dl, scale=0.08,
                                           workspace=workspace)
        w = satk.latent_rows_weights(q, cache, rows, lse, scale=0.08, counts=count, status=status)
        how = dict(kind="weights", scope="listed", row_ends=ends)
        loss, norm = satk.distill_loss(scores, ids, w, **how)
        return ids, out, w, loss, satk.distill_grad(scores, ids, w, norm, one, **how)
    table, req = i32([[0]]), i32([0] * T)
    workspace = torch.empty(satk.latent_workspace_bytes(H, dl), dtype=torch.uint8, device=DEV)
    first = True
    step()
    first = False
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (8, 9):
        scores.copy_(torch.randn(T, S, generator=gen(seed), device=DEV))
        want = [x.clone() for x in step()]
        for x in captured:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b)
        assert (captured[4][2] == 0).all() and captured[3][2] == 0
        # a row's gradient adds up to nothing: two distributions
        assert captured[4].double().sum(1).abs().max() < 1e-5
    assert int(status.item()) == 0
