"""The latent-cache entry points without a GPU: every refusal of the host
checks, with placeholder (never dereferenced) pointers, and the binding's own
checks on CPU tensors."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from sparse_attention_indexer_radix_gb300 import build as satk_build

OK, EINVAL, EUNSUPPORTED = 0, -1, -2
P = ctypes.c_void_p(4096)  # placeholder: never dereferenced by a rejected call
NULL = None
BF16, F16, F32 = 1, 2, 0
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="placeholder pointers only where no GPU can run a kernel")


@pytest.fixture(scope="module")
def lib():
    satk_build.build()
    return binding.lib()


def caller(f, ok):
    def call(**kw):
        assert set(kw) <= set(ok)
        return f(*{**ok, **kw}.values())
    return call


@no_gpu
def test_step_tables_rejects(lib):
    call = caller(lib.satk_step_tables, dict(
        ctx=P, new=P, R=4, W=2, rank=1, B=64, stride=64, free=P, n_free=10, table=P, ld=8,
        maxb=8, drafted=0, T=0x7fffffff, starts=P, lens=P, req=P, pos=P, ends=P, slots=P, used=P,
        st=NULL, stream=NULL))
    for name in ("ctx", "new", "free", "table", "starts", "lens", "req", "pos", "ends", "slots",
                 "used"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(R=-1), dict(W=0), dict(rank=2), dict(rank=-1), dict(B=0), dict(stride=-1),
               dict(n_free=-1), dict(n_free=2**31), dict(ld=7), dict(maxb=-1), dict(drafted=2),
               dict(T=-1), dict(T=2**31)):
        assert call(**kw) == EINVAL, kw
    assert call(R=8193) == EUNSUPPORTED


@no_gpu
def test_latent_store_rejects(lib):
    call = caller(lib.satk_latent_store, dict(
        x=P, ldx=128, tail=P, ldt=32, dt=BF16, T=4, dl=128, dr=32, w=P, eps=1e-6, cs=P, n=10,
        pos=P, il=0, slots=P, cache=P, rows=100, ldc=160, st=NULL, stream=NULL))
    for name in ("x", "tail", "pos", "slots", "cache"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=F32), dict(dt=9), dict(T=-1), dict(T=2**31), dict(dl=0), dict(dr=-2),
               dict(dr=31), dict(ldx=127), dict(ldt=31), dict(ldc=159), dict(rows=-1),
               dict(n=-1)):
        assert call(**kw) == EINVAL, kw
    assert call(dl=513, ldx=513, ldc=600) == EUNSUPPORTED
    assert call(dr=66, ldt=66, ldc=600) == EUNSUPPORTED
    assert call(T=0) == OK


def attend_args(extra):
    head = dict(q=P, dt=BF16, T=4, H=8, dl=128, dr=32, ldqt=8 * 160, ldqh=160, cache=P,
                rows=1000, ldc=160)
    end = dict(scale=0.1, out=P, ldot=8 * 128, ldoh=128, lse=NULL, ws=P, wsb=1 << 40, st=NULL,
               stream=NULL)
    return {**head, **extra, **end}


def attend_refusals(call):
    for name in ("q", "cache", "out", "ws"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=F32), dict(T=-1), dict(T=2**31), dict(H=0), dict(dl=0), dict(dr=-1),
               dict(ldqt=159), dict(ldqh=159), dict(ldc=159), dict(rows=-1), dict(ldot=127),
               dict(ldoh=127), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ws=ctypes.c_void_p(4104)), dict(wsb=0)):
        assert call(**kw) == EINVAL, kw
    assert call(dl=513, ldqh=1000, ldqt=10000, ldc=1000, ldoh=1000, ldot=10000) == EUNSUPPORTED
    assert call(dr=65, ldqh=1000, ldqt=10000, ldc=1000) == EUNSUPPORTED
    assert call(H=1025) == EUNSUPPORTED
    assert call(T=0) == OK


@no_gpu
def test_latent_attend_rejects(lib):
    call = caller(lib.satk_latent_attend, attend_args(dict(
        req=P, table=P, R=2, ldb=16, maxb=16, B=64, stride=64, ends=P, tree=P, words=2)))
    attend_refusals(call)
    for name in ("req", "table", "ends"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(R=-1), dict(ldb=15), dict(maxb=-1), dict(B=0), dict(stride=-1),
               dict(words=0)):
        assert call(**kw) == EINVAL, kw
    assert call(words=33) == EUNSUPPORTED


@no_gpu
def test_latent_attend_rows_rejects(lib):
    call = caller(lib.satk_latent_attend_rows, attend_args(dict(
        rowids=P, ldr=64, k=64, counts=P)))
    attend_refusals(call)
    assert call(rowids=NULL) == EINVAL
    assert call(k=0) == EINVAL
    assert call(ldr=63) == EINVAL


@no_gpu
def test_latent_attend_expanded_rejects(lib):
    call = caller(lib.satk_latent_attend_expanded, dict(
        q=P, dt=F16, T=4, H=8, dn=64, dr=32, ldqt=8 * 96, ldqh=96, k=P, S=9, ldks=8 * 64,
        ldkh=64, tail=P, ldt=32, v=P, dv=64, ldvs=8 * 64, ldvh=64, ts=P, ks=P, R=1, ends=P,
        scale=0.1, out=P, ldot=8 * 64, ldoh=64, lse=NULL, stream=NULL))
    for name in ("q", "k", "tail", "v", "ts", "ks", "ends", "out"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=F32), dict(T=-1), dict(T=2**31), dict(S=-1), dict(S=2**31), dict(R=-1),
               dict(H=0), dict(dn=0), dict(dr=-1), dict(dv=0), dict(ldqt=95), dict(ldqh=95),
               dict(ldks=63), dict(ldkh=63), dict(ldt=31), dict(ldvs=63), dict(ldvh=63),
               dict(ldot=63), dict(ldoh=63), dict(scale=float("nan"))):
        assert call(**kw) == EINVAL, kw
    assert call(H=1025) == EUNSUPPORTED
    assert call(dn=225) == EUNSUPPORTED
    assert call(dv=129) == EUNSUPPORTED
    assert call(T=0) == OK


@no_gpu
def test_latent_merge_rejects(lib):
    call = caller(lib.satk_latent_merge, dict(
        parts=P, dt=BF16, W=2, T=4, H=8, dv=128, ldw=4 * 8 * 128, ldt=8 * 128, ldh=128, lse=P,
        out=P, ldot=8 * 128, ldoh=128, lo=NULL, stream=NULL))
    for name in ("parts", "lse", "out"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=F32), dict(W=0), dict(T=-1), dict(T=2**31), dict(T=2**28), dict(H=0),
               dict(dv=0), dict(ldw=127), dict(ldt=127), dict(ldh=127), dict(ldot=127),
               dict(ldoh=127)):
        assert call(**kw) == EINVAL, kw
    assert call(W=65) == EUNSUPPORTED
    assert call(T=0) == OK


def test_workspace_bytes(lib):
    assert satk.latent_workspace_bytes(16, 512) > 0
    for bad in ((0, 512), (16, 0), (1025, 512), (16, 513)):
        assert satk.latent_workspace_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros(4, 8, 32, dtype=torch.bfloat16)
    c = torch.zeros(16, 32, dtype=torch.bfloat16)
    t = torch.zeros(4, 4, dtype=torch.int32)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.step_tables(i, i, i, t, tokens=4, block_size=4, stride_rows=4)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_store(c[:4], None, i, c)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_attend(x, c, i, t, i, block_size=4, stride_rows=4, latent_dim=16, scale=1.0)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_attend_rows(x, c, t, latent_dim=16, scale=1.0)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_attend_expanded(x, x, None, x, i, i, i, scale=1.0)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_merge(x[None], torch.zeros(1, 4, 8))
