"""Decode steps of one attention block: the serving operators together.

A batch of requests, each with its own low-rank adapter (or none), feeds one token per step through

  qkv  = X Wqkv^T + s_i (X A_i^T) B_i^T              LoraPlan
  q, k = rotate(norm(q)), rotate(norm(k)); k, v -> cache    qk_norm_rope
  o    = softmax(q K^T / sqrt(d)) V over the request's pages  PagedAttentionPlan
  y    = o Wo^T + s_i (o A'_i^T) B'_i^T              LoraPlan

The step is captured into one CUDA graph: adapters, positions, cache slots, block tables and lengths are device tensors that
it reads at every replay.  ``python examples/attention_block.py`` runs it on random weights, compares the last step with a plain
form of the whole sequence, and prints the time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_blackwell_gb300 as dg  # noqa: E402


class AttentionBlock:
    """Weights, cache and plans of one block for up to `batch` requests."""

    def __init__(self, batch, *, hidden=4096, heads=32, kv_heads=8, head_dim=128, rank=16, adapters=8, page=16, max_tokens=512, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(torch.bfloat16)  # noqa: E731
        self.batch, self.hidden, self.heads, self.kv_heads, self.head_dim, self.page = batch, hidden, heads, kv_heads, head_dim, page
        n_qkv, n_o = (heads + 2 * kv_heads) * head_dim, heads * head_dim
        self.w_qkv, self.w_o = r(n_qkv, hidden, scale=hidden ** -0.5), r(hidden, n_o, scale=n_o ** -0.5)
        self.a_qkv, self.b_qkv = r(adapters, rank, hidden, scale=hidden ** -0.5), r(adapters, n_qkv, rank, scale=0.2)
        self.a_o, self.b_o = r(adapters, rank, n_o, scale=n_o ** -0.5), r(adapters, hidden, rank, scale=0.2)
        self.lora_scale = 0.5 + torch.rand(adapters, generator=gen, device="cuda")
        self.q_norm, self.k_norm = 1 + r(head_dim, scale=0.1), 1 + r(head_dim, scale=0.1)
        self.rope = dg.rope_table(max_tokens, head_dim)
        # a pool of pages; every request gets its own, scattered over it
        width = -(-max_tokens // page)
        self.k_cache = torch.zeros(batch * width, page, kv_heads, head_dim, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.zeros_like(self.k_cache)
        self.block_table = torch.randperm(batch * width, generator=gen, device="cuda").to(torch.int32).view(batch, width)
        # one step's inputs and buffers
        self.x = torch.zeros(batch, hidden, dtype=torch.bfloat16, device="cuda")
        self.adapter = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
        self.positions = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.qkv = torch.empty(batch, n_qkv, dtype=torch.bfloat16, device="cuda")
        self.q = torch.empty(batch, heads, head_dim, dtype=torch.bfloat16, device="cuda")
        self.o, self.y = torch.empty_like(self.q), torch.empty_like(self.x)
        self.plan_qkv = dg.LoraPlan(batch, n_qkv, hidden, rank=rank, adapters=adapters)
        self.plan_o = dg.LoraPlan(batch, hidden, n_o, rank=rank, adapters=adapters)
        self.plan_attn = dg.PagedAttentionPlan(batch, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page)

    def step(self):
        """One token per request: x -> y, with positions[b] tokens of request b in the cache before."""
        h, g, d, page = self.heads, self.kv_heads, self.head_dim, self.page
        self.plan_qkv.run(self.x, self.w_qkv, self.a_qkv, self.b_qkv, self.adapter, self.qkv, scale=self.lora_scale)
        q = self.qkv[:, : h * d].unflatten(1, (h, d))
        k = self.qkv[:, h * d: (h + g) * d].unflatten(1, (g, d))
        v = self.qkv[:, (h + g) * d:].unflatten(1, (g, d))
        pages = self.block_table.gather(1, (self.positions // page).long()[:, None])[:, 0]
        slots = pages * page + self.positions % page
        dg.qk_norm_rope(q, k, self.positions, self.rope, q_weight=self.q_norm, k_weight=self.k_norm, q_out=self.q, v=v, k_cache=self.k_cache,
                        v_cache=self.v_cache, slots=slots)
        self.plan_attn.run(self.q, self.k_cache, self.v_cache, self.block_table, self.positions + 1, self.o)
        self.plan_o.run(self.o.flatten(1), self.w_o, self.a_o, self.b_o, self.adapter, self.y, scale=self.lora_scale)
        return self.y

    def capture(self):
        """A graph of step(); replay() runs it on the current contents of x, adapter, positions and block_table."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()                      # plans and kernels are set up outside the capture
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def close(self):
        for plan in (self.plan_qkv, self.plan_o, self.plan_attn):
            plan.close()

    def plain(self, xs):
        """The outputs of the last of the steps xs [steps, batch, hidden], computed over the whole sequences in fp32."""
        h, g, d = self.heads, self.kv_heads, self.head_dim
        steps = xs.shape[0]

        def project(x, w, a, b):
            y = x @ w.float().T
            for i, j in enumerate(self.adapter.tolist()):
                if j >= 0:
                    y[:, i] += self.lora_scale[j] * ((x[:, i] @ a[j].float().T) @ b[j].float().T)
            return y

        def norm_rotate(t, weight):
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
            c, s = self.rope[:steps, 0][:, None, None], self.rope[:steps, 1][:, None, None]
            a, b = t.chunk(2, -1)
            return torch.cat((a * c - b * s, a * s + b * c), -1)

        qkv = project(xs.float(), self.w_qkv, self.a_qkv, self.b_qkv)
        q = norm_rotate(qkv[..., : h * d].unflatten(-1, (h, d)), self.q_norm)[-1]
        k = norm_rotate(qkv[..., h * d: (h + g) * d].unflatten(-1, (g, d)), self.k_norm).repeat_interleave(h // g, 2)
        v = qkv[..., (h + g) * d:].unflatten(-1, (g, d)).repeat_interleave(h // g, 2)
        p = torch.softmax(torch.einsum("bhd,sbhd->bhs", q, k) * d ** -0.5, -1)
        o = torch.einsum("bhs,sbhd->bhd", p, v).flatten(1)
        return project(o[None], self.w_o, self.a_o, self.b_o)[0]


def run(batch=16, steps=40, **sizes):
    """Decodes `steps` tokens per request; returns (relative error of the last step against the plain form, us per step)."""
    block = AttentionBlock(batch, max_tokens=max(steps, 16), **sizes)
    block.adapter.copy_(torch.arange(batch, device="cuda") % (block.a_qkv.shape[0] + 1) - 1)
    graph = block.capture()
    gen = torch.Generator(device="cuda").manual_seed(1)
    xs = torch.randn(steps, batch, block.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    for t in range(steps):
        block.x.copy_(xs[t])
        block.positions.fill_(t)
        graph.replay()
    want = block.plain(xs)
    error = ((block.y.float() - want).norm() / want.norm()).item()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    block.close()
    return error, start.elapsed_time(end) / 20 * 1e3


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    dg.build()
    error, us = run(args.batch, args.steps)
    print("last step against the plain form: relative error %.2g; %.1f us per step of %d requests" % (error, us, args.batch))
    # bf16 activations between the operators: a few roundings of 2^-9 each
    sys.exit(0 if error < 0.02 else 1)
