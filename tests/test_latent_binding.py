"""What the binding checks before it calls the library, on CPU tensors: the
queries for devices and streams are stubbed and the calls go to a stand-in
that records them."""
from __future__ import annotations

import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding

BF16 = torch.bfloat16


class Library:
    """Takes any entry point's call, records its name and arguments, returns 0
    (a size from the workspace query)."""

    def __init__(self):
        self.calls, self.devices = [], []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            self.devices.append(torch.cuda.current_device())
            return 64 if name == "satk_latent_workspace_bytes" else 0
        return entry


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(binding, "lib", lambda: L)
    monkeypatch.setattr(binding, "_device_of", lambda *ts: 0)
    monkeypatch.setattr(binding, "_need_cuda", lambda *ts: 0)
    monkeypatch.setattr(binding, "_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_stream_on", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    return L


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def step_tables(table=None, **kw):
    return satk.step_tables(i32(4), i32(4), i32(8), i32(4, 6) if table is None else table,
                            tokens=4, block_size=4, stride_rows=4, **kw)


def latent_store(**kw):
    return satk.latent_store(torch.zeros(4, 32, dtype=BF16), None, i32(4),
                             torch.zeros(16, 32, dtype=BF16), **kw)


def latent_attend(table=None, **kw):
    return satk.latent_attend(torch.zeros(4, 2, 32, dtype=BF16), torch.zeros(16, 32, dtype=BF16),
                              i32(4), i32(4, 6) if table is None else table, i32(4), block_size=4,
                              stride_rows=4, latent_dim=16, scale=1.0, **kw)


def latent_attend_rows(**kw):
    return satk.latent_attend_rows(torch.zeros(4, 2, 32, dtype=BF16),
                                   torch.zeros(16, 32, dtype=BF16), i32(4, 6), latent_dim=16,
                                   scale=1.0, **kw)


def dcp_rescue_select(**kw):
    return satk.dcp_rescue_select(i32(2, 4, 33), torch.zeros(2, 4, 64, dtype=BF16), i32(4),
                                  i32(4, 16), 16, recv=i32(64), **kw)


def dcp_emit_rows(table=None, **kw):
    return satk.dcp_emit_rows(i32(4, 6), 1, 0, i32(4), i32(4, 6) if table is None else table, 4, 4,
                              **kw)


CALLS = [step_tables, latent_store, latent_attend, latent_attend_rows, dcp_rescue_select,
         dcp_emit_rows]


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_status_is_a_whole_word(call, library, monkeypatch):
    """Kernels OR bits into four bytes of it: no other type, and not the
    stand-in address of a tensor without elements."""
    monkeypatch.setattr(binding, "rescue_recv_words", lambda T, n, k: 64)
    word = i32(1)
    call(status=word)
    assert any(getattr(a, "value", a) == word.data_ptr() for a in library.calls[-1][1])
    library.calls.clear()
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(8, dtype=torch.bool)[1:],
                torch.zeros(2, dtype=torch.float32)):
        with pytest.raises(satk.SatkError, match="status"):
            call(status=bad)
    assert not [c for c in library.calls if c[0] != "satk_latent_workspace_bytes"]
    try:
        call(status=i32(0))
    except satk.SatkError:
        return
    assert binding._EMPTY_BATCH_PTR not in [getattr(a, "value", a) for a in library.calls[-1][1]]


@pytest.mark.parametrize("call", [step_tables, latent_attend, dcp_emit_rows],
                         ids=lambda f: f.__name__)
def test_max_blocks_stays_within_the_table(call, library):
    """Columns past a table that is a slice of a wider one belong to others, and
    past the last row's they may not exist."""
    table = i32(4, 10)[:, 2:8]
    for ok in (None, 0, 5, 6):
        call(table=table, max_blocks=ok)
    library.calls.clear()
    for bad in (7, 8, 10):
        with pytest.raises(satk.SatkError, match="max_blocks"):
            call(table=table, max_blocks=bad)
    assert not [c for c in library.calls if c[0] != "satk_latent_workspace_bytes"]


def topk_rows(**kw):
    return satk.topk_rows(torch.zeros(4, 32), 8, **kw)


def dcp_pack():
    return satk.dcp_pack(torch.zeros(4, 64, dtype=BF16), i32(4, 32))


def dcp_topk_pack():
    return satk.dcp_topk_pack(torch.zeros(4, 64, dtype=BF16), 32)


def dcp_merge_select():
    return satk.dcp_merge_select(i32(2, 4, 33), 16, packed=True)


def latent_attend_expanded():
    x = torch.zeros(4, 2, 32, dtype=BF16)
    return satk.latent_attend_expanded(x, x, None, x, i32(2), i32(2), i32(4), scale=1.0)


def latent_merge():
    return satk.latent_merge(torch.zeros(2, 4, 2, 32, dtype=BF16), torch.zeros(2, 4, 2))


@pytest.mark.parametrize("call", [*CALLS, topk_rows, dcp_pack, dcp_topk_pack, dcp_merge_select,
                                  latent_attend_expanded, latent_merge], ids=lambda f: f.__name__)
def test_calls_run_on_their_tensors_device(call, library, monkeypatch):
    """Tensors on device 1 while device 0 is current: the library (launches,
    kernel attributes, the SM count behind the workspace's size) is entered
    with device 1 current, and device 0 is current again afterwards."""
    current = [0]

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *error):
            current.pop()

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(binding, "_device_of", lambda *ts: 1)
    monkeypatch.setattr(binding, "_need_cuda", lambda *ts: 1)
    monkeypatch.setattr(binding, "rescue_recv_words", lambda T, n, k: 64)
    call()
    assert library.devices and set(library.devices) == {1}
    assert current == [0]
    library.devices.clear()
    monkeypatch.setattr(binding, "_device_of", lambda *ts: 0)
    monkeypatch.setattr(binding, "_need_cuda", lambda *ts: 0)
    call()
    assert set(library.devices) == {0}
