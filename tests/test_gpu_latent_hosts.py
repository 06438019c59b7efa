"""Host-side conditions of the latent-cache calls on the GPU: several threads
that call at once, and batch sizes at the edges of shared memory."""
from __future__ import annotations

import sys
import threading

import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from test_gpu_latent import BF16, DEV, expanded_case, gen, i32, latent_rows, tables_oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


def selected(seed, D, latent):
    g = gen(seed)
    cache = latent_rows(g, 256, D, BF16)
    q = torch.randn(2, 64, D, generator=g, device=DEV).to(BF16)
    rows = torch.randint(0, 256, (2, 70), generator=g, device=DEV).int()
    size = satk.latent_workspace_bytes(64, latent)
    kw = dict(workspace=torch.empty(size, dtype=torch.uint8, device=DEV),
              out=torch.empty(2, 64, latent, dtype=BF16, device=DEV),
              lse=torch.empty(2, 64, device=DEV))
    return lambda: satk.latent_attend_rows(q, cache, rows, latent_dim=latent, scale=0.1, **kw)


def expanded(seed, dn, dr, dv):
    g = gen(seed)
    q, k, tail, v, ts, ks, ends = expanded_case(g, BF16, 2, dn, dr, dv, [70], [30])
    args = (q, k, tail, v, i32(ts), i32(ks), i32(ends))
    kw = dict(out=torch.empty(70, 2, dv, dtype=BF16, device=DEV),
              lse=torch.empty(70, 2, device=DEV))
    return lambda: satk.latent_attend_expanded(*args, scale=0.1, **kw)


def tables(requests):
    zero, one = i32(np.zeros(requests)), i32(np.ones(requests))
    free, table = i32(np.arange(requests)), i32(np.full((requests, 2), -1))
    out = satk.StepTables(*(i32(np.zeros(n)) for n in (requests + 1, requests, *[requests] * 4, 1)))
    return lambda: tuple(satk.step_tables(zero, one, free, table, tokens=requests, block_size=4,
                                          stride_rows=4, out=out))


def paged(seed, D, latent):
    g = gen(seed)
    cache = latent_rows(g, 256, D, BF16)
    q = torch.randn(2, 16, D, generator=g, device=DEV).to(BF16)
    req, table, ends = i32([0, 1]), i32([[0, 2], [1, 3]]), i32([100, 37])
    return lambda: satk.latent_attend(q, cache, req, table, ends, block_size=64, stride_rows=64,
                                      latent_dim=latent, scale=0.1)


@pytest.mark.parametrize("make,args", [(selected, (3, 576, 512)), (paged, (7, 160, 128)),
                                       (expanded, (5, 128, 64, 128)), (tables, (8192,))])
def test_first_call_of_a_thread(make, args):
    """A call that is a host thread's first use of CUDA."""
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
    assert not errors, errors
    for x, y in zip(want, got):
        assert torch.equal(x, y)


class Recorder:
    """Passes calls on to the library and keeps the last one."""

    def __init__(self, library):
        self.library = library

    def __getattr__(self, name):
        f = getattr(self.library, name)

        def entry(*args):
            self.last = f, args
            return f(*args)
        return entry


@pytest.mark.parametrize("make,wide,narrow", [
    (selected, (3, 576, 512), (4, 64, 64)),
    (expanded, (5, 192, 64, 128), (6, 32, 0, 32)),
    (tables, (8192,), (6200,))])
def test_threads_with_wide_and_narrow_calls(make, wide, narrow):
    """Two host threads, each on its own stream and buffers, call one kernel
    with much and with little shared memory, over and over: neither takes it
    from the other between its setting and the launch."""
    calls = [make(*wide), make(*narrow)]
    want = [tuple(x.clone() for x in f()) for f in calls]
    torch.cuda.synchronize()
    begin, failed, got = threading.Barrier(2), [0, 0], [None, None]

    def work(i):
        stream, recorder = torch.cuda.Stream(), Recorder(binding.lib())
        with torch.cuda.stream(stream):
            with binding.routed_to(recorder):
                got[i] = calls[i]()
            f, args = recorder.last
            begin.wait()
            for _ in range(20000):
                failed[i] += f(*args) != 0
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    before = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(before)
    torch.cuda.synchronize()
    assert failed == [0, 0]
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("R", [4096, 4097, 6112, 6113, 6144, 6145, 8192])
def test_tables_at_the_edges_of_shared_memory(R):
    """The scan's arrays (8 bytes a request) next to the kernel's fixed ones:
    below, at and above what a block gets without asking for more."""
    rng = np.random.RandomState(R)
    ctx, new = rng.randint(0, 9, R), rng.randint(0, 3, R)
    free, table = rng.permutation(R * 3)[:2 * R].astype(np.int32), np.zeros((R, 3), np.int32)
    want = tables_oracle(ctx, new, free, table, 2 * R, 4, 4, 1, 0, False)
    dt = i32(table)
    got = satk.step_tables(i32(ctx), i32(new), i32(free), dt, tokens=2 * R, block_size=4,
                           stride_rows=4)
    assert np.array_equal(dt.cpu().numpy(), want[0])
    for name, x, y in zip(satk.StepTables._fields, got, want[1:8]):
        assert x.cpu().tolist() == list(y), name
