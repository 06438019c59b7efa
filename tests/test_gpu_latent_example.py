"""examples/latent_step.py, whose steps chain the latent-cache operators with
the indexer's selection, against 64-bit attention over the tokens they say
they attend to."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir, "examples",
                    "latent_step.py")
U = 2.0**-8  # half a bf16 step


@pytest.fixture(scope="module")
def example():
    from sparse_attention_indexer_radix_gb300 import build as satk_build
    satk_build.build()
    spec = importlib.util.spec_from_file_location("latent_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def global_row(layer, r, p):
    """The cached row of request r's global token p."""
    rank, l = p % layer.W, p // layer.W
    block = int(layer.tables[rank][r, l // layer.block])
    return layer.caches[rank][block * layer.block + l % layer.block].double()


def check(out, lse, q, keys, dl, scale, roundings):
    s = (q.double() @ keys.T) * scale
    want = torch.logsumexp(s, 1)
    p = torch.exp(s - want[:, None])
    v = keys[:, :dl]
    tol = roundings * U * (p @ v.abs()) + 1e-4
    assert ((out.double() - p @ v).abs() <= tol).all()
    assert ((lse.double() - want).abs() <= 1e-4).all()


def test_runs_as_a_script(example, capsys):
    example.main()
    assert "verify" in capsys.readouterr().out


@pytest.mark.parametrize("W", [1, 2, 4])
def test_decode_steps(example, W):
    layer = example.Layer(W=W, seed=W)
    layer.prompt([200, 37, 1, 150, 90])
    for _ in range(2):
        d = layer.decode_step()
    lens = layer.lens.tolist()
    for r in range(layer.R):
        ids = [g for g in d["ids"][r].tolist() if g >= 0]
        assert len(ids) == min(layer.k, lens[r]) == len(set(ids)) and max(ids) < lens[r]
        keys = torch.stack([global_row(layer, r, g) for g in ids])
        # weights, a rank's result and the join: a rounding each
        check(d["out"][r], d["lse"][r], d["q"][r], keys, layer.dl, layer.scale, 3)
    assert int(layer.status.item()) == 0


def test_verify_trees(example):
    layer = example.Layer(W=1, seed=7)
    layer.prompt([100, 20, 33, 64, 1])
    parents = [-1, 0, 0, 1, 2, 2, 5, -1] + list(range(7, 35))
    t = layer.verify(parents)
    n, lens = len(parents), layer.lens.tolist()
    for r in range(layer.R):
        for i in range(n):
            at = list(range(lens[r])) + [lens[r] + b for b in range(n) if t["bits"][i] >> b & 1]
            keys = torch.stack([global_row(layer, r, g) for g in at])
            check(t["out"][r * n + i], t["lse"][r * n + i], t["q"][r * n + i], keys, layer.dl,
                  layer.scale, 2)
    assert int(layer.status.item()) == 0


def test_expanded_and_absorbed_forms_agree(example):
    """The prompts' expanded attention equals the absorbed one: queries through
    the key projection, results through the value projection."""
    layer = example.Layer(W=1, seed=9)
    p = layer.prompt([70, 130, 5, 33, 64])
    dl, H, hd = layer.dl, layer.H, 64
    w_k, w_v = (w.double().view(dl, H, hd) for w in (p["w_k"], p["w_v"]))
    q = p["q"].double()
    starts = p["starts"].tolist()
    latent, tail = p["rows"][:, :dl].double(), p["rows"][:, dl:].double()
    for r in range(layer.R):
        a, b = starts[r], starts[r + 1]
        absorbed = torch.einsum("thd,lhd->thl", q[a:b, :, :hd], w_k)
        s = torch.einsum("thl,sl->ths", absorbed, latent[a:b])
        s = (s + torch.einsum("thd,sd->ths", q[a:b, :, hd:], tail[a:b])) * p["scale"]
        s = s.masked_fill(torch.triu(torch.ones(b - a, b - a, dtype=torch.bool, device=s.device), 1)
                          [:, None], float("-inf"))
        w = torch.softmax(s, 2)
        want = torch.einsum("ths,sl,lhd->thd", w, latent[a:b], w_v)
        # keys and values were rounded once each on their way: 2-norms
        off = (p["out"][a:b].double() - want).norm() / want.norm()
        assert off <= 4 * U, off
