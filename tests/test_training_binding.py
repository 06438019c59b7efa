"""What the binding checks and passes on for the training calls, on CPU tensors: the
calls go to a stand-in that records them."""
from __future__ import annotations

import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from test_latent_binding import BF16, i32, library  # noqa: F401


def distill(**kw):
    rows = kw.pop("rows", 4)
    return dict(logits=torch.zeros(rows, 50), ids=i32(rows, 8), teacher=torch.zeros(rows, 8), **kw)


def test_distill_arguments(library):  # noqa: F811
    loss, lse = satk.distill_loss(**distill(kind="probs", scope="listed", temperature=0.5, k=5,
                                            row_ends=i32(4)))
    assert loss.shape == lse.shape == (4,) and loss.dtype == torch.float32
    name, args = library.calls[-1]
    assert name == "satk_distill_loss"
    assert args[1:5] == (0, 4, 50, 50) and args[7:9] == (8, 5) and args[10:15] == (0, 8, 2, 1, 0.5)


@pytest.mark.parametrize("dloss,step", [(torch.zeros(4), 1), (torch.zeros(1), 0),
                                        (torch.zeros(()), 0), (torch.zeros(()).expand(4), 0)])
def test_one_dloss_or_one_a_row(library, dloss, step):  # noqa: F811
    out = satk.distill_grad(lse=torch.zeros(4), dloss=dloss, **distill())
    assert out.shape == (4, 50)
    assert library.calls[-1][1][17] == step


def test_one_row_has_free_strides(library):  # noqa: F811
    a = dict(distill(rows=1))
    a["logits"] = torch.zeros(1, 100)[:, ::1][:, :50]
    satk.distill_loss(**a)
    assert library.calls[-1][1][2:5] == (1, 50, 50)


@pytest.mark.parametrize("kw", [dict(kind=None), dict(kind="logit"), dict(scope="ROW"), dict(k=9),
                                dict(row_ends=i32(3)), dict(row_ends=torch.zeros(4)),
                                dict(loss=torch.zeros(3)), dict(lse=torch.zeros(4, dtype=BF16))])
def test_distill_refusals(library, kw):  # noqa: F811
    with pytest.raises(satk.SatkError):
        satk.distill_loss(**distill(**kw))
    assert not library.calls


def weights(**kw):
    a = dict(q=torch.zeros(4, 2, 32, dtype=BF16), cache=torch.zeros(16, 40, dtype=BF16), rows=i32(4, 9),
             lse=torch.zeros(4, 2), scale=1.0)
    return satk.latent_rows_weights(**{**a, **kw})


def test_weights_arguments(library):  # noqa: F811
    assert weights(k=7).shape == (4, 7)
    name, args = library.calls[-1]
    assert name == "satk_latent_rows_weights"
    assert args[1:7] == (1, 4, 2, 32, 64, 32) and args[8:10] == (16, 40) and args[11:13] == (9, 7)
    out = torch.zeros(4, 12)
    assert weights(out=out) is out and library.calls[-1][1][17] == 12


@pytest.mark.parametrize("kw", [dict(status=torch.zeros(1)), dict(status=i32(0)), dict(counts=i32(3)),
                                dict(out=torch.zeros(4, 8)), dict(lse=torch.zeros(2, 4)),
                                dict(cache=torch.zeros(16, 31, dtype=BF16)), dict(rows=i32(4, 9).t())])
def test_weights_refusals(library, kw):  # noqa: F811
    with pytest.raises(satk.SatkError):
        weights(**kw)
    assert not library.calls


def grad(**kw):
    T, S, H = 4, 6, 2

    def z(*shape):
        return torch.zeros(*shape, dtype=BF16)
    a = dict(dout=z(T, H, 16), q=z(T, H, 48), k=z(S, H, 32), tail=z(S, 16), v=z(S, H, 16),
             out=z(T, H, 16), lse=torch.zeros(T, H), token_starts=i32(3), key_starts=i32(3),
             row_ends=i32(T), scale=0.5)
    return satk.latent_attend_expanded_grad(**{**a, **kw})


def test_grad_arguments(library):  # noqa: F811
    dq, dk, dtail, dv = grad(workspace=torch.zeros(64, dtype=torch.uint8))
    assert (dq.shape, dk.shape, dtail.shape, dv.shape) == ((4, 2, 48), (6, 2, 32), (6, 16), (6, 2, 16))
    name, args = library.calls[-1]
    assert name == "satk_latent_attend_expanded_grad"
    assert args[5:10] == (1, 4, 2, 32, 16) and args[13] == 6 and args[24] == 2 and args[-2] == 64
    assert grad(tail=None, q=torch.zeros(4, 2, 32, dtype=BF16),
                workspace=torch.zeros(64, dtype=torch.uint8))[2] is None
    name, args = library.calls[-1]
    assert args[9] == 0 and args[16] is None


@pytest.mark.parametrize("kw", [dict(tail=None), dict(dtail=torch.zeros(6, 8, dtype=BF16)),
                                dict(key_starts=i32(2)), dict(dlse=torch.zeros(4, 2, dtype=BF16)),
                                dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0])])
def test_grad_refusals(library, kw):  # noqa: F811
    with pytest.raises(satk.SatkError):
        grad(**kw)
    assert not [c for c in library.calls if c[0] == "satk_latent_attend_expanded_grad"]
