"""Steps of a sparse-attention layer over a latent cache, end to end.

    python examples/latent_step.py

W ranks hold the tokens of a few requests in turn (global token p on rank
p % W); here they are only W caches on one GPU.  Every layer input (latents,
queries, indexer scores) is random; the plain matrix products around the
calls (projections, indexer scores) are torch's.

prompt():      the prompts' tokens are written to the caches (step_tables,
               latent_store) and attend to each other in the expanded form
               (latent_attend_expanded).
decode_step(): one new token a request: step_tables and latent_store on every
               rank, the indexer's top-k over all ranks (dcp_topk_pack,
               dcp_merge_select), each rank's cache rows of it
               (dcp_emit_rows), attention over them (latent_attend_rows) and
               the join of the ranks (latent_merge).
verify():      a drafted tree of tokens a request: their rows are written
               behind the context and each token attends to the context and
               its ancestors (latent_attend with a tree; one rank).
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import sparse_attention_indexer_radix_gb300 as satk  # noqa: E402


class Layer:
    """One layer's caches, block tables and position table on W ranks."""

    def __init__(self, requests=5, W=2, heads=16, latent=128, tail=32, block=16, capacity=512,
                 k=64, dtype=torch.bfloat16, device="cuda:0", seed=0):
        self.R, self.W, self.H, self.dl, self.dr = requests, W, heads, latent, tail
        self.block, self.k, self.dtype, self.dev = block, k, dtype, device
        self.gen = torch.Generator(device=device).manual_seed(seed)
        width = -(-(-(-capacity // W)) // block)
        blocks = requests * width
        self.tables = [torch.full((requests, width), -1, dtype=torch.int32, device=device)
                       for _ in range(W)]
        self.free = [torch.randperm(blocks, generator=self.gen, device=device).int()
                     for _ in range(W)]
        self.caches = [torch.zeros(blocks * block, latent + tail, dtype=dtype, device=device)
                       for _ in range(W)]
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        inv = 10000.0 ** (-torch.arange(0, tail, 2, dtype=torch.float64) / tail)
        angle = torch.arange(capacity, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.norm = torch.rand(latent, generator=self.gen, device=device) + 0.5
        self.scale = 1.0 / math.sqrt(latent + tail)

    def random(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.dev).to(self.dtype)

    def write(self, new, drafted=False):
        """Slots for `new` tokens of each request (int32 [R]) and their rows in
        the caches.  Returns every rank's StepTables and the rows' latents and
        rotated tails as they were written."""
        T = int(new.sum())
        latent, tail = self.random(T, self.dl), self.random(T, self.dr)
        steps = []
        for r in range(self.W):
            t = satk.step_tables(self.lens, new, self.free[r], self.tables[r], tokens=T,
                                 block_size=self.block, stride_rows=self.block, W=self.W,
                                 dcp_rank=r, drafted=drafted, status=self.status)
            self.free[r] = self.free[r][int(t.blocks_used):]
            satk.latent_store(latent, tail, t.slots, self.caches[r], weight=self.norm,
                              cos_sin=self.cos_sin, positions=t.positions, status=self.status)
            steps.append(t)
        self.lens = self.lens + new
        return steps, latent, tail

    def prompt(self, lengths, heads_dim=64):
        """The prompts' causal attention in the expanded form: per-head keys and
        values from the latents that the cache holds."""
        new = torch.tensor(lengths, dtype=torch.int32, device=self.dev)
        steps, _, _ = self.write(new)
        T = int(new.sum())
        rows = torch.empty(T, self.dl + self.dr, dtype=self.dtype, device=self.dev)
        for r, t in enumerate(steps):  # the rows back in token order
            held = t.slots >= 0
            rows[held] = self.caches[r][t.slots[held].long()]
        w_k = self.random(self.dl, self.H * heads_dim) / math.sqrt(self.dl)
        w_v = self.random(self.dl, self.H * heads_dim) / math.sqrt(self.dl)
        k = (rows[:, :self.dl] @ w_k).view(T, self.H, heads_dim)
        v = (rows[:, :self.dl] @ w_v).view(T, self.H, heads_dim)
        q = self.random(T, self.H, heads_dim + self.dr)
        starts = steps[0].token_starts
        ends = steps[0].positions + 1  # all ranks' keys are here: global ends
        scale = 1.0 / math.sqrt(heads_dim + self.dr)
        out, lse = satk.latent_attend_expanded(q, k, rows[:, self.dl:], v, starts, starts, ends,
                                               scale=scale)
        return dict(q=q, rows=rows, w_k=w_k, w_v=w_v, starts=starts, scale=scale, out=out, lse=lse)

    def decode_step(self):
        """One token a request over its k best cached tokens of all ranks."""
        new = torch.ones(self.R, dtype=torch.int32, device=self.dev)
        steps, _, _ = self.write(new)
        q = self.random(self.R, self.H, self.dl + self.dr)
        # the indexer's scores of each rank's local tokens
        width = self.tables[0].shape[1] * self.block
        scores = self.random(self.W, self.R, width)
        n = self.k
        packed = torch.stack([satk.dcp_topk_pack(scores[r], n, row_ends=steps[r].row_ends)
                              for r in range(self.W)])
        ids = satk.dcp_merge_select(packed, self.k, packed=True, status=self.status)
        parts, lses, rows = [], [], []
        for r in range(self.W):
            at, count = satk.dcp_emit_rows(ids, self.W, r, steps[r].req_id, self.tables[r],
                                           self.block, self.block, status=self.status)
            out, lse = satk.latent_attend_rows(q, self.caches[r], at, counts=count,
                                               latent_dim=self.dl, scale=self.scale,
                                               status=self.status)
            parts.append(out)
            lses.append(lse)
            rows.append((at, count))
        out, lse = satk.latent_merge(torch.stack(parts), torch.stack(lses))
        return dict(q=q, ids=ids, scores=scores, out=out, lse=lse)

    def verify(self, parents):
        """A drafted tree a request (parents[i] < i, or -1 for a root) over its
        context: one rank's caches.  The tokens' rows stay behind the context;
        the lengths do not move."""
        assert self.W == 1, "a tree's bits count local tokens: one rank"
        n = len(parents)
        lens = self.lens
        new = torch.full((self.R,), n, dtype=torch.int32, device=self.dev)
        steps, _, _ = self.write(new, drafted=True)
        self.lens = lens  # nothing is accepted here
        bits = []
        for i, p in enumerate(parents):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        words = -(-n // 32)
        tree = torch.tensor([[b >> (32 * w) & 0xffffffff for w in range(words)] for b in bits],
                            dtype=torch.int64, device=self.dev)
        tree = torch.where(tree >= 2**31, tree - 2**32, tree).int().repeat(self.R, 1)
        q = self.random(self.R * n, self.H, self.dl + self.dr)
        t = steps[0]
        out, lse = satk.latent_attend(q, self.caches[0], t.req_id, self.tables[0], t.row_ends,
                                      block_size=self.block, stride_rows=self.block,
                                      latent_dim=self.dl, scale=self.scale, tree=tree,
                                      status=self.status)
        return dict(q=q, bits=bits, out=out, lse=lse)


def main():
    layer = Layer()
    p = layer.prompt([200, 37, 1, 150, 90])
    print("prompt   out", tuple(p["out"].shape), "mean lse %.3f" % p["lse"].mean().item())
    for _ in range(3):
        d = layer.decode_step()
    print("decode   out", tuple(d["out"].shape), "mean lse %.3f" % d["lse"].mean().item())
    single = Layer(W=1, seed=1)
    single.prompt([100, 20, 33, 64, 1])
    t = single.verify([-1, 0, 0, 1, 2, 2, 5])
    print("verify   out", tuple(t["out"].shape), "mean lse %.3f" % t["lse"].mean().item())
    for x in (layer, single):
        assert int(x.status.item()) == 0, "a status bit was raised"


if __name__ == "__main__":
    main()
