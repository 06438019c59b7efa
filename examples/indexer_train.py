"""Training steps around a sparse-attention layer: the indexer that selects, the
prompt attention, and a student of another model's top logits.

    python examples/indexer_train.py

Every layer input is random; the plain matrix products (projections, the
indexer's scores) and their gradients are torch's.

index_step():     the indexer's scores of a sequence select rows of its latent
                  cache (topk_rows, dcp_emit_rows); the attention over them
                  (latent_attend_rows) says how much weight each got
                  (latent_rows_weights), and the indexer is trained towards
                  that (distill_loss, distill_grad over the selected columns).
attention_step(): prompts attend to each other in the expanded form
                  (latent_attend_expanded); the gradient of the result goes
                  back to queries, keys, the shared tail and values
                  (latent_attend_expanded_grad) and on to the projections.
student_step():   a student's logits against the top entries of a teacher's
                  (topk_rows, distill_loss, distill_grad in the logits' place).
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), os.pardir))
import sparse_attention_indexer_radix_gb300 as satk  # noqa: E402


class Trainer:
    """One layer's weights and one sequence's latent cache in shuffled blocks."""

    def __init__(self, tokens=300, heads=16, latent=128, tail=32, block=16, k=64, index_heads=4,
                 index_dim=32, width=64, vocab=1000, dtype=torch.bfloat16, device="cuda:0", seed=0):
        self.T, self.H, self.dl, self.dr, self.block, self.k = tokens, heads, latent, tail, block, k
        self.dtype, self.dev = dtype, device
        self.gen = torch.Generator(device=device).manual_seed(seed)
        blocks = -(-tokens // block)
        self.table = torch.randperm(blocks, generator=self.gen, device=device).int()[None].contiguous()
        rows = self.table[0].long()[:, None] * block + torch.arange(block, device=device)
        self.cache = torch.empty(blocks * block, latent + tail, dtype=dtype, device=device)
        self.keys = self.normal(tokens, latent + tail)
        self.cache[rows.flatten()[:tokens]] = self.keys
        self.ends = torch.arange(1, tokens + 1, dtype=torch.int32, device=device)
        self.request = torch.zeros(tokens, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

        def weight(*shape):
            w = torch.randn(*shape, generator=self.gen, device=device) / math.sqrt(shape[0])
            return w.requires_grad_()
        self.w_index_q = weight(latent + tail, index_heads * index_dim)
        self.w_index_k = weight(latent + tail, index_dim)
        self.w_index = weight(latent + tail, index_heads)
        self.index_heads = index_heads
        self.w_q = weight(latent, heads * (width + tail))
        self.w_k, self.w_v = weight(latent, heads * width), weight(latent, heads * width)
        self.width = width
        self.w_vocab = weight(latent, vocab)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=self.dev).to(self.dtype)

    def index_scores(self):
        """The indexer's scores [T, T] in float32: relu of each index head's products,
        weighted by the token."""
        x = self.keys.float()
        q = (x @ self.w_index_q).view(self.T, self.index_heads, -1)
        products = torch.relu(torch.einsum("thd,sd->ths", q, x @ self.w_index_k))
        return torch.einsum("ths,th->ts", products, x @ self.w_index)

    def index_step(self, rate=0.0):
        q = self.normal(self.T, self.H, self.dl + self.dr)
        scale = 1.0 / math.sqrt(self.dl + self.dr)
        scores = self.index_scores()
        values = scores.detach()
        ids = satk.topk_rows(values, self.k, row_ends=self.ends)
        rows, count = satk.dcp_emit_rows(ids, 1, 0, self.request, self.table, self.block, self.block,
                                         status=self.status)
        out, lse = satk.latent_attend_rows(q, self.cache, rows, counts=count, latent_dim=self.dl,
                                           scale=scale, status=self.status)
        weights = satk.latent_rows_weights(q, self.cache, rows, lse, scale=scale, counts=count,
                                           status=self.status)
        how = dict(kind="weights", scope="listed", row_ends=self.ends)
        loss, norm = satk.distill_loss(values, ids, weights, **how)
        each = torch.full((1,), 1.0 / self.T, device=self.dev)
        scores.backward(satk.distill_grad(values, ids, weights, norm, each, **how))
        parameters = [self.w_index_q, self.w_index_k, self.w_index]
        return dict(q=q, ids=ids, count=count, out=out, weights=weights, loss=loss.mean(),
                    grads=self.step(parameters, rate))

    def attention_step(self, lengths, rate=0.0):
        """Prompts whose lengths add up to the sequence's, each on its own."""
        starts = torch.tensor([0] + lengths, device=self.dev).cumsum(0).int()
        ends = torch.cat([torch.arange(1, n + 1) for n in lengths]).int().to(self.dev)
        latent, tail = self.keys[:, :self.dl], self.keys[:, self.dl:].contiguous()
        q, k, v = ((latent @ w.to(self.dtype)).view(self.T, self.H, -1)
                   for w in (self.w_q, self.w_k, self.w_v))
        scale = 1.0 / math.sqrt(self.width + self.dr)
        with torch.no_grad():
            out, lse = satk.latent_attend_expanded(q, k, tail, v, starts, starts, ends, scale=scale)
            dout = self.normal(self.T, self.H, self.width)
            dq, dk, dtail, dv = satk.latent_attend_expanded_grad(dout, q, k, tail, v, out, lse, starts,
                                                                 starts, ends, scale=scale)
        torch.autograd.backward([q, k, v], [dq, dk, dv])
        return dict(out=out, dout=dout, dtail=dtail, starts=starts, scale=scale,
                    grads=self.step([self.w_q, self.w_k, self.w_v], rate))

    def student_step(self, temperature=2.0, rate=0.0):
        logits = (self.keys[:, :self.dl] @ self.w_vocab.to(self.dtype)).float()
        teacher = logits.detach() + self.normal(*logits.shape).float()
        ids = satk.topk_rows(teacher, 20)
        top = teacher.gather(1, ids.long())
        values = logits.detach().clone()
        loss, norm = satk.distill_loss(values, ids, top, temperature=temperature)
        each = torch.full((1,), temperature ** 2 / self.T, device=self.dev)
        grad = satk.distill_grad(values, ids, top, norm, each, temperature=temperature, out=values)
        logits.backward(grad)
        return dict(ids=ids, top=top, loss=loss.mean(), grads=self.step([self.w_vocab], rate))

    @staticmethod
    def step(parameters, rate):
        """A step down the gradients, which are handed back and cleared."""
        grads = [p.grad for p in parameters]
        with torch.no_grad():
            for p in parameters:
                p.sub_(rate * p.grad)
                p.grad = None
        return grads


def main():
    t = Trainer()
    for _ in range(3):
        print("indexer   divergence %.4f" % t.index_step(rate=0.1)["loss"].item())
    a = t.attention_step([100, 37, 1, 162], rate=0.01)
    print("attention |gradients|", " ".join("%.3f" % g.norm().item() for g in a["grads"]))
    for _ in range(3):
        print("student   divergence %.4f" % t.student_step(rate=1.0)["loss"].item())
    assert int(t.status.item()) == 0, "a status bit was raised"


if __name__ == "__main__":
    main()
