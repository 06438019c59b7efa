"""examples/indexer_train.py, whose steps chain the training operators with the
selection and the attention, against 64-bit steps that torch differentiates."""
from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir, "examples",
                    "indexer_train.py")
U = 2.0**-8  # half a bf16 step


@pytest.fixture(scope="module")
def example():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()
    spec = importlib.util.spec_from_file_location("indexer_train", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def near(got, want, rel):
    assert (got.double() - want).norm() <= rel * want.norm(), \
        ((got.double() - want).norm() / want.norm()).item()


def test_runs_as_a_script(example, capsys):
    example.main()
    assert "student" in capsys.readouterr().out


@pytest.mark.parametrize("tokens,heads,k", [(300, 16, 64), (129, 3, 200), (1, 20, 8)])
def test_index_step(example, tokens, heads, k):
    t = example.Trainer(tokens=tokens, heads=heads, k=k, seed=1)
    r = t.index_step()
    keys = t.keys.double()
    w = [p.detach().double().requires_grad_() for p in (t.w_index_q, t.w_index_k, t.w_index)]
    q = (keys @ w[0]).view(tokens, t.index_heads, -1)
    scores = torch.einsum("ths,th->ts", torch.relu(torch.einsum("thd,sd->ths", q, keys @ w[1])),
                          keys @ w[2])
    total, scale = 0.0, 1.0 / math.sqrt(t.dl + t.dr)
    for i in range(tokens):
        ids = [j for j in r["ids"][i].tolist() if j >= 0]
        assert len(ids) == min(k, i + 1) == int(r["count"][i]) and max(ids) <= i
        p = torch.softmax(r["q"][i].double() @ keys[ids].T * scale, 1)
        near(r["weights"][i, :len(ids)], p.mean(0), 1e-4)
        near(r["out"][i], p @ keys[ids][:, :t.dl], 3 * U)
        p = p.mean(0)
        total = total + (p * (torch.log(p) - torch.log_softmax(scores[i, ids], 0))).sum() / tokens
    total.backward()
    # the scores, the weights and the torch products are float32
    assert abs(r["loss"].item() - total.item()) <= 1e-4 * (1 + abs(total.item()))
    for got, x in zip(r["grads"], w):
        assert (got.double() - x.grad).norm() <= 1e-3 * x.grad.norm() + 1e-6
    assert int(t.status.item()) == 0


def test_attention_step(example):
    t = example.Trainer(seed=2)
    r = t.attention_step([100, 37, 1, 162])
    latent, tail = t.keys[:, :t.dl].double(), t.keys[:, t.dl:].double().requires_grad_()
    w = [p.detach().to(t.dtype).double().requires_grad_() for p in (t.w_q, t.w_k, t.w_v)]
    q, k, v = ((latent @ x).view(t.T, t.H, -1) for x in w)
    total = 0.0
    for a, b in zip(r["starts"].tolist()[:-1], r["starts"].tolist()[1:]):
        key = torch.cat([k[a:b], tail[a:b, None].expand(-1, t.H, -1)], 2)
        s = torch.einsum("thd,shd->hts", q[a:b], key) * r["scale"]
        s = s.masked_fill(torch.ones(b - a, b - a, dtype=torch.bool, device=s.device).triu(1),
                          -math.inf)
        out = torch.einsum("hts,shd->thd", torch.softmax(s, 2), v[a:b])
        near(r["out"][a:b], out.detach(), 6 * U)
        total = total + (out * r["dout"][a:b].double()).sum()
    total.backward()
    # queries, keys and values are rounded on their way in, weights and scores'
    # gradients between, gradients on their way out
    for got, x in zip(r["grads"], w):
        near(got, x.grad, 8 * U)
    near(r["dtail"], tail.grad, 8 * U)


def test_student_step(example):
    t = example.Trainer(seed=3)
    r = t.student_step(temperature=2.0)
    x, w = t.keys[:, :t.dl], t.w_vocab.detach()
    # (the logits as the student has them: rounded to bfloat16)
    logits = (x @ w.to(t.dtype)).double().requires_grad_()
    p = torch.softmax(r["top"].double() / 2.0, 1)
    log_q = torch.log_softmax(logits / 2.0, 1).gather(1, r["ids"].long())
    loss = (p * (torch.log(p) - log_q)).sum(1).mean()
    (loss * 4.0).backward()
    assert abs(r["loss"].item() - loss.item()) <= 1e-5 * (1 + abs(loss.item()))
    # the gradient goes back through bfloat16 products
    near(r["grads"][0], x.double().T @ logits.grad, 4 * U)
