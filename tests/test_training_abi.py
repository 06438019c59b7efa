"""The training entry points without a GPU: every refusal of the host checks, with
placeholder (never dereferenced) pointers, and the binding's own checks."""
from __future__ import annotations

import ctypes

import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from sparse_attention_indexer_radix_gb300 import binding
from test_latent_abi import BF16, EINVAL, EUNSUPPORTED, F16, F32, NULL, OK, P, caller, lib, no_gpu  # noqa: F401

DISTILL = dict(x=P, dt=BF16, rows=4, cols=100, ld=100, ends=NULL, ids=P, ldi=8, k=8, teacher=P,
               tdt=F32, ldt=8, kind=0, scope=0, tau=1.0)


def distill_refusals(call):
    for name in ("x", "ids", "teacher"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=3), dict(dt=-1), dict(tdt=7), dict(rows=-1), dict(rows=2**31), dict(cols=-1),
               dict(cols=2**31, ld=2**31), dict(ld=99), dict(ldi=7), dict(ldt=7), dict(k=0),
               dict(k=4097, ldi=5000, ldt=5000), dict(kind=-1), dict(kind=3), dict(scope=-1),
               dict(scope=2), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
               dict(tau=float("inf")), dict(tau=1e-45)):
        assert call(**kw) == EINVAL, kw
    assert call(rows=0) == OK


@no_gpu
def test_distill_loss_rejects(lib):  # noqa: F811
    call = caller(lib.satk_distill_loss, dict(**DISTILL, loss=P, lse=P, stream=NULL))
    distill_refusals(call)
    assert call(loss=NULL) == call(lse=NULL) == EINVAL


@no_gpu
def test_distill_grad_rejects(lib):  # noqa: F811
    grad = ctypes.c_void_p(8192)
    call = caller(lib.satk_distill_grad, dict(**DISTILL, lse=P, dloss=P, step=1, grad=grad, ldg=100,
                                              stream=NULL))
    distill_refusals(call)
    for kw in (dict(lse=NULL), dict(dloss=NULL), dict(grad=NULL), dict(step=2), dict(step=-1),
               dict(ldg=99), dict(grad=P, ldg=101)):
        assert call(**kw) == EINVAL, kw
    assert call(cols=0, ld=0) == OK


@no_gpu
def test_rows_weights_rejects(lib):  # noqa: F811
    call = caller(lib.satk_latent_rows_weights, dict(
        q=P, dt=BF16, T=4, H=8, D=160, ldqt=8 * 160, ldqh=160, cache=P, rows=1000, ldc=160,
        rowids=P, ldr=64, k=64, counts=NULL, scale=0.1, lse=P, out=P, ldo=64, st=NULL, stream=NULL))
    for name in ("q", "cache", "rowids", "lse", "out"):
        assert call(**{name: NULL}) == EINVAL
    for kw in (dict(dt=F32), dict(dt=9), dict(T=-1), dict(T=2**31), dict(H=0), dict(D=0), dict(k=0),
               dict(rows=-1), dict(ldqt=159), dict(ldqh=159), dict(ldc=159), dict(ldr=63),
               dict(ldo=63), dict(scale=float("nan")), dict(scale=float("-inf"))):
        assert call(**kw) == EINVAL, kw
    assert call(H=1025) == EUNSUPPORTED
    assert call(D=577, ldqt=9000, ldqh=600, ldc=600) == EUNSUPPORTED
    assert call(T=0) == OK


@no_gpu
def test_expanded_grad_rejects(lib):  # noqa: F811
    call = caller(lib.satk_latent_attend_expanded_grad, dict(
        dout=P, lddt=512, lddh=64, dlse=NULL, q=P, dt=F16, T=4, H=8, dn=64, dr=32, ldqt=8 * 96,
        ldqh=96, k=P, S=9, ldks=512, ldkh=64, tail=P, ldt=32, v=P, dv=64, ldvs=512, ldvh=64, ts=P,
        ks=P, R=1, ends=P, scale=0.1, out=P, ldot=512, ldoh=64, lse=P, gq=P, ldgqt=8 * 96, ldgqh=96,
        gk=P, ldgks=512, ldgkh=64, gt=P, ldgt=32, gv=P, ldgvs=512, ldgvh=64, ws=P, wsb=1 << 40,
        stream=NULL))
    for name in ("dout", "q", "k", "tail", "v", "ts", "ks", "ends", "out", "lse", "gq", "gk", "gt",
                 "gv", "ws"):
        assert call(**{name: NULL}) == EINVAL, name
    for kw in (dict(dt=F32), dict(T=-1), dict(T=2**31), dict(S=-1), dict(S=2**31), dict(R=-1),
               dict(H=0), dict(dn=0), dict(dr=-1), dict(dv=0), dict(scale=float("nan")),
               dict(ws=ctypes.c_void_p(4104)), dict(wsb=0), dict(lddt=63), dict(lddh=63),
               dict(ldqt=95), dict(ldqh=95), dict(ldks=63), dict(ldkh=63), dict(ldt=31),
               dict(ldvs=63), dict(ldvh=63), dict(ldot=63), dict(ldoh=63), dict(ldgqt=95),
               dict(ldgqh=95), dict(ldgks=63), dict(ldgkh=63), dict(ldgt=31), dict(ldgvs=63),
               dict(ldgvh=63)):
        assert call(**kw) == EINVAL, kw
    assert call(H=1025) == EUNSUPPORTED
    assert call(dn=225, ldqh=257, ldqt=9000, ldgqh=257, ldgqt=9000, ldkh=225, ldks=9000, ldgkh=225,
                ldgks=9000) == EUNSUPPORTED
    assert call(dv=129) == EUNSUPPORTED
    assert call(T=0, S=0) == OK


def test_grad_workspace_bytes(lib):  # noqa: F811
    f = satk.latent_expanded_grad_workspace_bytes
    assert f(4096, 8192, 1, 16, 64) >= 4096 * 16 * 8 + 8192 * 16 * 64 * 4
    assert f(0, 0, 0, 1, 0) >= 0
    for bad in ((-1, 1, 1, 1, 0), (2**31, 1, 1, 1, 0), (1, -1, 1, 1, 0), (1, 1, -1, 1, 0),
                (1, 1, 1, 0, 0), (1, 1, 1, 1025, 0), (1, 1, 1, 1, -1), (1, 1, 1, 1, 257)):
        assert f(*bad) == 0


def test_binding_refuses_cpu_tensors():
    i, f = torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4)
    x = torch.zeros(4, 8, 32, dtype=torch.bfloat16)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.distill_loss(f, i, f)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.distill_grad(f, i, f, f[0], f[0])
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_rows_weights(x, x[:, 0], i, f, scale=1.0)
    with pytest.raises(satk.SatkError, match="CUDA"):
        satk.latent_attend_expanded_grad(x, x, x, None, x, x, f, i[0], i[0], i[0], scale=1.0)


def test_every_training_entry_point_is_exported():
    for name in ("distill_loss", "distill_grad", "latent_rows_weights",
                 "latent_attend_expanded_grad", "latent_expanded_grad_workspace_bytes"):
        assert name in satk.__all__ and callable(getattr(satk, name))
        assert "satk_" + name in binding.EXPORTS
