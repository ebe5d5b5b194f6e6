"""One feed-forward block with its residual norm: the operators of a training step and of decode steps together.

Training, in 16 bits, forward and backward:

  h, n = x + residual, norm(x + residual)            add_rms_norm
  H    = act(n Wg^T) * (n Wu^T)                      GatedPlan
  y    = H Wd^T                                      Plan
  dH   = dy Wd, dWd = dy^T H                         Plan, operands as they lie in memory
  dn, dWg, dWu                                       GatedPlan.backward
  dx, dw                                             add_rms_norm_backward

The next block's norm leaves its result in 8 bits with scales for the projection after it, a block-scaled or an MXFP8 product.

Decode steps of up to 16 requests run on the same block with weights in 4 bits (add_rms_norm, int4_matmul as the gated pair,
int4_matmul), captured into one CUDA graph.  ``python examples/feed_forward.py`` runs all of it on random weights, compares with
plain forms and prints times.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_blackwell_gb300 as dg  # noqa: E402
from dense_gemm_blackwell_gb300 import inputs  # noqa: E402


def activation(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh" if kind == "gelu_tanh" else "none")


class FeedForward:
    """Weights and plans of one block for steps of exactly `tokens` tokens; sizes are multiples of 8."""

    def __init__(self, tokens, *, hidden=4096, features=8192, kind="silu", dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen, device="cuda") * scale).to(dtype)  # noqa: E731
        self.tokens, self.hidden, self.features, self.kind = tokens, hidden, features, kind
        self.w_norm = (1 + 0.2 * r(hidden)).to(dtype)
        self.w_gate_up, self.w_down = r(2 * features, hidden, scale=hidden ** -0.5), r(hidden, features, scale=features ** -0.5)
        self.H = torch.empty(tokens, features, dtype=dtype, device="cuda")
        self.gate_up = torch.empty(tokens, 2 * features, dtype=dtype, device="cuda")
        self.y = torch.empty(tokens, hidden, dtype=dtype, device="cuda")
        self.dH = torch.empty_like(self.H)
        self.dw_down = torch.empty(hidden, features, device="cuda")
        code = {torch.bfloat16: dg.GEMM_BF16, torch.float16: dg.GEMM_F16}[dtype]
        self.gated = dg.GatedPlan(tokens, features, hidden, activation=kind, dtype=code, gradients=True, dtype_dw=dg.GEMM_F32)
        self.down = dg.Plan(dg.make_desc(tokens, hidden, features, dtype_a=code, dtype_d=code))
        # dH [tokens, features] = dy [tokens, hidden] Wd [hidden, features];  dWd [hidden, features] = dy^T H
        self.down_dH = dg.Plan(dg.make_desc(tokens, features, hidden, dtype_a=code, dtype_d=code, major_b=dg.GEMM_MN_MAJOR))
        self.down_dw = dg.Plan(dg.make_desc(hidden, features, tokens, dtype_a=code, major_a=dg.GEMM_MN_MAJOR, major_b=dg.GEMM_MN_MAJOR))

    def forward(self, x, residual):
        """(y, h): the block's output and the residual that goes on beside it."""
        self.n, _, self.h = dg.add_rms_norm(x, self.w_norm, residual=residual)
        self.gated.run(self.n, self.w_gate_up, self.H, gate_up=self.gate_up)
        self.down.run(self.H, self.w_down, self.y)
        return self.y, self.h

    def backward(self, dy, dh=None):
        """Gradients of forward(): of x and of the residual alike, and of the three weights (fp32); dh is what reaches h."""
        self.down_dH.run(dy, self.w_down, self.dH)
        self.down_dw.run(dy, self.H, self.dw_down)
        dn, dw_gate_up = self.gated.backward(self.dH, self.n, self.w_gate_up, self.gate_up)
        dx, dw_norm = dg.add_rms_norm_backward(dn, self.h, self.w_norm, d_sum=dh, out=dn)
        return dx, dw_norm, dw_gate_up, self.dw_down

    def close(self):
        for plan in (self.gated, self.down, self.down_dH, self.down_dw):
            plan.close()

    def plain(self, x, residual, w_norm=None, w_gate_up=None, w_down=None):
        """(y, h) in 64 bits, from the block's weights or those given."""
        w_norm, w_gate_up, w_down = (own.double() if w is None else w for own, w in (
            (self.w_norm, w_norm), (self.w_gate_up, w_gate_up), (self.w_down, w_down)))
        h = x.double() + residual.double()
        n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w_norm
        g, u = (n @ w_gate_up.T).chunk(2, -1)
        return (activation(g, self.kind) * u) @ w_down.T, h


def project(y, h, w_norm, codes, scales, mode):
    """The next block's norm and projection in 8 bits: norm(y + h) W^T, W as E4M3 codes with scales."""
    a, sa, _ = dg.add_rms_norm(y, w_norm, residual=h, scale_mode=mode)
    if mode == dg.GEMM_SCALE_BLOCK_1x128_128x128:
        return dg.matmul(a, codes, scale_a=sa, scale_b=scales, out_dtype=torch.bfloat16)
    out = torch.empty(a.shape[0], codes.shape[0], dtype=torch.bfloat16, device=a.device)
    with dg.Plan(dg.make_desc(*out.shape, a.shape[1], dtype_a=dg.GEMM_E4M3, dtype_d=dg.GEMM_BF16, scale_mode=mode)) as plan:
        plan.run_mx(a, codes, out, sa, scales)
        torch.cuda.synchronize()             # before the plan goes
    return out


class Decode4Bit:
    """Decode steps of `batch` requests on the block's weights in 4 bits."""

    def __init__(self, block, batch, group=128):
        self.group, self.kind, self.w_norm = group, block.kind, block.w_norm
        self.gate_up, self.down = dg.int4_quantize(block.w_gate_up, group), dg.int4_quantize(block.w_down, group, symmetric=False)
        self.x = torch.zeros(batch, block.hidden, dtype=block.w_norm.dtype, device="cuda")
        self.residual = torch.zeros_like(self.x)

    def step(self):
        """x, residual -> y; the residual becomes their sum."""
        n, _, _ = dg.add_rms_norm(self.x, self.w_norm, residual=self.residual, sum_out=self.residual)
        codes, scales, zeros = self.gate_up
        H = dg.int4_matmul(n, codes, scales, zeros=zeros, group=self.group, activation=self.kind)
        codes, scales, zeros = self.down
        self.y = dg.int4_matmul(H, codes, scales, zeros=zeros, group=self.group)
        return self.y

    def capture(self):
        """A graph of step(); replay() runs it on the current contents of x and residual, and leaves its result in y."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def weights(self, packed):
        """A packed weight matrix as 64-bit numbers."""
        codes, scales, zeros = packed
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double()
        wide = lambda t: t.double().repeat_interleave(self.group, 1)[:, : q.shape[1]]  # noqa: E731
        return wide(scales) * (q - (8.0 if zeros is None else wide(zeros)))


def relative(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def train(tokens, steps=0, **sizes):
    """One training step; returns ({output or gradient: relative error against 64 bits}, us per step over `steps` more)."""
    block = FeedForward(tokens, **sizes)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, residual, dy, dh = (torch.randn(tokens, block.hidden, generator=gen, device="cuda").to(block.H.dtype) for _ in range(4))
    y, h = block.forward(x, residual)
    grads = block.backward(dy, dh)
    leaves = [t.double().requires_grad_() for t in (x, block.w_norm, block.w_gate_up, block.w_down)]
    want_y, want_h = block.plain(leaves[0], residual, *leaves[1:])
    want = torch.autograd.grad([want_y, want_h], leaves, [dy.double(), dh.double()])
    errors = {"y": relative(y, want_y.detach()), "h": relative(h, want_h.detach())}
    for name, got, ref in zip(("dx", "dw_norm", "dw_gate_up", "dw_down"), grads, want):
        errors[name] = relative(got, ref)
    us = 0.0
    if steps:
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(steps):
            block.forward(x, residual)
            block.backward(dy, dh)
        end.record()
        torch.cuda.synchronize()
        us = start.elapsed_time(end) / steps * 1e3
    block.close()
    return errors, us


def next_projection(tokens, columns, mode, **sizes):
    """Forward pass, then the next block's norm and projection in 8 bits; relative error against 64 bits on the same weights."""
    block = FeedForward(tokens, **sizes)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, residual = (torch.randn(tokens, block.hidden, generator=gen, device="cuda").to(block.H.dtype) for _ in range(2))
    w = torch.randn(columns, block.hidden, generator=gen, device="cuda") * block.hidden ** -0.5
    if mode == dg.GEMM_SCALE_BLOCK_1x128_128x128:
        codes, scales = (t.cuda() for t in inputs.block_quantize_e4m3(w.cpu(), 128))
        wide = scales.double().repeat_interleave(128, 0)[:columns].repeat_interleave(128, 1)[:, : block.hidden]
    else:
        # a power of two for every 32 columns, as the norm writes it
        amax = torch.nn.functional.pad(w, (0, -block.hidden % 32)).unflatten(1, (-1, 32)).abs().amax(2)
        exponent = torch.ceil(torch.log2(amax / 448)).clamp(-126, 127)
        wide = torch.exp2(exponent).double().repeat_interleave(32, 1)[:, : block.hidden]
        codes = (w / wide.float()).to(torch.float8_e4m3fn)
        scales = inputs.pack_scales_tiled((exponent + 127).to(torch.uint8).cpu()).cuda()
    y, h = block.forward(x, residual)
    got = project(y, h, block.w_norm, codes, scales, mode)
    want_y, want_h = block.plain(x, residual)
    s = want_y + want_h
    n = s * torch.rsqrt(s.square().mean(-1, keepdim=True) + 1e-6) * block.w_norm.double()
    error = relative(got, n @ (codes.double() * wide).T)
    block.close()
    return error


def decode(batch, steps=8, group=128, **sizes):
    """`steps` replays of a captured decode step; (largest relative error of a step against 64 bits, us per step)."""
    block = FeedForward(8, **sizes)
    dec = Decode4Bit(block, batch, group)
    w_gate_up, w_down = dec.weights(dec.gate_up), dec.weights(dec.down)
    graph = dec.capture()
    gen = torch.Generator(device="cuda").manual_seed(3)
    worst = 0.0
    for _ in range(steps):
        dec.x.copy_(torch.randn(batch, block.hidden, generator=gen, device="cuda"))
        dec.residual.copy_(torch.randn(batch, block.hidden, generator=gen, device="cuda"))
        want_y, want_h = block.plain(dec.x, dec.residual, None, w_gate_up, w_down)
        graph.replay()
        worst = max(worst, relative(dec.y, want_y), relative(dec.residual, want_h))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    block.close()
    return worst, start.elapsed_time(end) / 20 * 1e3


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--batch", type=int, default=8)
    args = ap.parse_args()
    dg.build()
    errors, us = train(args.tokens, steps=10)
    print("training step of %d tokens: %.0f us; relative errors %s" % (
        args.tokens, us, ", ".join("%s %.2g" % e for e in errors.items())))
    eight = [next_projection(args.tokens, 4096, mode) for mode in (dg.GEMM_SCALE_BLOCK_1x128_128x128, dg.GEMM_SCALE_MX_E8M0_32)]
    print("next projection in 8 bits: relative error %.2g (block scales), %.2g (MXFP8)" % tuple(eight))
    error, us = decode(args.batch)
    print("decode step of %d requests, 4-bit weights: %.1f us; relative error %.2g" % (args.batch, us, error))
    # 16-bit activations between the operators, half a step of 2^-8 each, twelve of them; half a step of E4M3, 2^-4, once
    sys.exit(0 if max(*errors.values(), error) < 12 * 2.0 ** -8 and max(eight) < 2.0 ** -4 + 12 * 2.0 ** -8 else 1)
