"""GPU: the example's feed-forward block runs the operators together, in training, with 8-bit and with 4-bit products.

Tolerances are in the norm of a whole output and count roundings to 16 bits, each at most half a step, u = eps / 2 relative, beside
which fp32 sums do not show.  h: 1.  y: h and n reach the product of two projections twice, then H and y: 6.  Gradients: G and U
carry h, n and their own rounding (3 each), then dH, d_gate_up, dn, h in the norm's backward pass and the result: 12 at most.
Codes of E4M3 are half a step of 2^-4 off; weights enter the 64-bit form as the codes stand for them.
"""
import importlib.util
import os

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
SIZES = [
    (1, dict(hidden=256, features=512)),
    (77, dict(hidden=520, features=712, kind="gelu")),
    (130, dict(hidden=1000, features=1544, kind="gelu_tanh", dtype=torch.float16)),
    (640, dict(hidden=1024, features=2048)),
]


@pytest.fixture(scope="module")
def example():
    dg.build()
    spec = importlib.util.spec_from_file_location("feed_forward", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def half_step(sizes):
    return torch.finfo(sizes.get("dtype", torch.bfloat16)).eps / 2


@pytest.mark.parametrize("tokens,sizes", SIZES)
def test_training_step_matches_the_formula(example, tokens, sizes):
    errors, _ = example.train(tokens, **sizes)
    for name, error in errors.items():
        assert error < {"h": 1, "y": 6}.get(name, 12) * half_step(sizes), (name, errors)


@pytest.mark.parametrize("tokens,sizes", SIZES[1:])
def test_gradients_match_differences(example, tokens, sizes):
    """Along a gradient g / |g| the loss <y, dy> + <h, dh> in 64 bits grows by |g|; central differences of step e are e^2 off."""
    block = example.FeedForward(tokens, **sizes)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, residual, dy, dh = (torch.randn(tokens, block.hidden, generator=gen, device="cuda").to(block.H.dtype) for _ in range(4))
    block.forward(x, residual)
    grads = [g.double() for g in block.backward(dy, dh)]
    leaves = [t.double() for t in (x, block.w_norm, block.w_gate_up, block.w_down)]

    def loss(i, step):
        at = [t + step * grads[i] / grads[i].norm() if j == i else t for j, t in enumerate(leaves)]
        y, h = block.plain(at[0], residual, *at[1:])
        return ((y * dy.double()).sum() + (h * dh.double()).sum()).item()

    for i, g in enumerate(grads):
        slope = (loss(i, 1e-4) - loss(i, -1e-4)) / 2e-4
        assert abs(slope / g.norm().item() - 1) < 12 * half_step(sizes), i
    block.close()


@pytest.mark.parametrize("mode", [dg.GEMM_SCALE_BLOCK_1x128_128x128, dg.GEMM_SCALE_MX_E8M0_32])
@pytest.mark.parametrize("tokens,columns,sizes", [(5, 256, dict(hidden=512, features=512)), (200, 384, dict(hidden=1024, features=1544, kind="gelu"))])
def test_next_projection_in_8_bits(example, tokens, columns, sizes, mode):
    assert example.next_projection(tokens, columns, mode, **sizes) < 2.0 ** -4 + 12 * half_step(sizes)


@pytest.mark.parametrize("batch,group,sizes", [
    (1, 128, dict(hidden=256, features=512)),
    (7, 64, dict(hidden=520, features=712, kind="gelu_tanh")),
    (16, 32, dict(hidden=1000, features=1544, dtype=torch.float16))])
def test_decode_steps_with_4_bit_weights(example, batch, group, sizes):
    error, _ = example.decode(batch, 3, group, **sizes)
    assert error < 6 * half_step(sizes)


def test_captured_training_step(example):
    """The whole step in one graph, replayed on new inputs, gives what the calls give."""
    block = example.FeedForward(96, hidden=512, features=768)
    gen = torch.Generator(device="cuda").manual_seed(6)
    new = lambda: [torch.randn(96, 512, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(4)]  # noqa: E731
    held = new()

    def step():
        y, h = block.forward(held[0], held[1])
        return (y, h) + block.backward(held[2], held[3])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(2):
        for t, s in zip(held, new()):
            t.copy_(s)
        want = [t.clone() for t in step()]
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        for got, ref in zip(out, want):
            assert torch.equal(got, ref)
    torch.cuda.synchronize()
    block.close()
