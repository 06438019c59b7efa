"""Refusals of the training entry points at the edges of their numbers, without a GPU."""
from __future__ import annotations

import ctypes

import pytest

from test_latent_abi import EINVAL, NULL, OK, P, caller, lib, no_gpu  # noqa: F401
from test_training_abi import DISTILL


@no_gpu
@pytest.mark.parametrize("tau", [4e-39, 3e-39, 1e-40])
def test_temperatures_whose_inverse_overflows_in_log2(lib, tau):  # noqa: F811
    """Scores are scaled by log2(e) / temperature: refused where that is infinite (of
    equal scores it would make NaN), taken where it is not."""
    grad = ctypes.c_void_p(8192)
    loss = caller(lib.satk_distill_loss, dict(**DISTILL, loss=P, lse=P, stream=NULL))
    back = caller(lib.satk_distill_grad, dict(**DISTILL, lse=P, dloss=P, step=1, grad=grad, ldg=100,
                                              stream=NULL))
    for call in (loss, back):
        assert call(tau=tau, rows=0) == EINVAL
        for taken in (4.3e-39, 1e-30, 1e30):
            assert call(tau=taken, rows=0) == OK
