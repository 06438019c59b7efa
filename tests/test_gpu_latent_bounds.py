"""Values at the ends of their ranges in the latent-cache calls: starts beyond
the tokens, scores near the ends of fp32, values that are not finite."""
from __future__ import annotations


import numpy as np
import pytest
import torch

import sparse_attention_indexer_radix_gb300 as satk
from test_gpu_latent import BF16, DEV, expanded_case, expanded_check, gen, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()


@pytest.mark.parametrize("dn", [64, 20])  # tensor cores, and the form for any width
@pytest.mark.parametrize("first,last", [(0, 2**31 - 1), (5, 2**31 - 1), (0, 2**31 - 9), (7, 300),
                                        (-2**31, 2**31 - 1)])
def test_expanded_starts_beyond_the_tokens(dn, first, last):
    """A last start past the tokens ends the request at the last token; tokens
    before the first start have empty rows."""
    T, H, dv = 150, 2, 32
    q, k, _, v, _, ks, ends = expanded_case(gen(81), BF16, H, dn, 0, dv, [T], [10])
    guard = torch.full((T + 64, H, dv), 3.0, dtype=BF16, device=DEV)
    lse_guard = torch.full((T + 64, H), 3.0, device=DEV)
    o, lse = satk.latent_attend_expanded(q, k, None, v, i32([first, last]), i32(ks), i32(ends),
                                         scale=0.2, out=guard[32:-32], lse=lse_guard[32:-32])
    begin = max(first, 0)
    assert torch.all(o[:begin] == 0) and torch.all(torch.isneginf(lse[:begin]))
    expanded_check(q, k, None, v, np.array([begin, T]), ks, ends, o, lse, 0.2)
    for x in (guard, lse_guard):
        assert torch.all(x[:32] == 3.0) and torch.all(x[-32:] == 3.0)
