"""GPU: the gated pair of projections against a 64-bit form: the kernel for few tokens and every tile of the pipeline, odd and ragged
sizes, padded rows, what the backward pass keeps, streams, graphs and two plans at once; and the gradients against the formula and
against differences."""
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: dg.GEMM_BF16, torch.float16: dg.GEMM_F16}
PAIR, LONE = dg.GEMM_FLAG_CTA_GROUP_2, dg.GEMM_FLAG_CTA_GROUP_1


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def rows(t, n, kind, seed, scale=1.0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = -(-n // 8) * 8 + pad
    return (torch.randn(t, ld, generator=gen, device="cuda") * scale).to(kind)[:, :n]


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")


def half_step(kind):
    return torch.finfo(kind).eps / 2


def sums_error(a, b, k):
    """Bound on an fp32 sum of k products: at most k steps of 2^-23 (the tensor core may truncate) of the magnitudes' sum."""
    return (a.double().abs() @ b.double().abs().T) * (min(k, 4096) * 2.0 ** -23)


def check_forward(x, w, act, out, gate_up=None):
    f, kind, k = w.shape[0] // 2, x.dtype, x.shape[1]
    both = x.double() @ w.double().T
    g, u = both[:, :f], both[:, f:]
    err = sums_error(x, w, k)
    dg_, du = err[:, :f], err[:, f:]
    a = act64(g, act)
    want = a * u
    least = 2.0 ** -25 if kind == torch.float16 else 0.0
    # the activations' slopes are under 1.13; the activation itself is computed to 2^-19 of |g|
    bound = 1.13 * dg_ * (u.abs() + du) + a.abs() * du + g.abs() * u.abs() * 2.0 ** -19 + want.abs() * half_step(kind) * (1 + 2.0 ** -8) + least
    assert ((out.double() - want).abs() <= bound).all(), ((out.double() - want).abs() - bound).max().item()
    if gate_up is not None:
        assert ((gate_up.double() - both).abs() <= err + (both.abs() + err) * half_step(kind) + least).all()


def run(t, f, k, kind, act, *, keep=False, pad=0, **plan):
    x, w = rows(t, k, kind, 1, pad=pad), rows(2 * f, k, kind, 2, 1.5 * k ** -0.5, pad=2 * pad)
    store = torch.full((t + 2, f + 16), 7.0, dtype=kind, device="cuda")
    out = store[1: t + 1, :f]
    kept = torch.full((t + 1, 2 * f + 8), 3.0, dtype=kind, device="cuda")
    gate_up = kept[:t, : 2 * f] if keep else None
    with dg.GatedPlan(t, f, k, activation=act, dtype=CODE[kind], ldx=x.stride(0) if t > 1 else 0 or -(-k // 8) * 8, ldw=w.stride(0),
                      ldh=f + 16, ld_gate_up=2 * f + 8, **plan) as p:
        assert p.run(x, w, out, gate_up) is out
        assert p.sync_status()[0] == dg.GEMM_OK
        info = p.info
        check_forward(x, w, act, out, gate_up)
        first = out.clone()
        out.fill_(float("nan"))
        p.run(x, w, out, gate_up)        # a second launch of the plan: fresh partials and flags
        assert p.sync_status()[0] == dg.GEMM_OK
        assert torch.equal(out, first)
    assert (store[0] == 7).all() and (store[-1] == 7).all() and (store[:, f:] == 7).all()
    assert (kept[t:] == 3).all() and (kept[:, 2 * f:] == 3).all()
    return info


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,f,k,act", [(1, 8, 1, "silu"), (1, 4096, 2048, "silu"), (2, 24, 63, "gelu"), (4, 1000, 1001, "gelu_tanh"), (7, 264, 65, "silu"),
                                       (8, 16, 4096, "gelu"), (9, 328, 333, "silu"), (16, 2048, 4096, "gelu_tanh"), (16, 40, 8200, "silu")])
def test_decode(t, f, k, act, kind):
    assert run(t, f, k, kind, act, keep=t % 2 == 1).few_tiles == 1


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,f,k,act", [(17, 8, 1, "silu"), (17, 136, 64, "gelu"), (96, 1024, 2048, "silu"), (127, 264, 130, "gelu_tanh"), (128, 64, 1000, "silu"),
                                       (129, 1544, 72, "gelu"), (300, 520, 1001, "silu"), (777, 1544, 1001, "gelu"), (1024, 4096, 1024, "gelu_tanh")])
def test_batches(t, f, k, act, kind):
    info = run(t, f, k, kind, act, keep=t % 2 == 1, pad=8)
    assert info.few_tiles == (t <= 128)      # none of these is wide enough for the pipeline to take 97 tokens


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("flags,tile,t,f,k,ctas", [
    (LONE, 128, 200, 200, 320, 0), (LONE, 256, 200, 328, 320, 0), (LONE, 512, 200, 600, 320, 0), (PAIR, 128, 300, 200, 320, 0),
    (PAIR, 256, 300, 328, 320, 0), (PAIR, 512, 300, 1000, 320, 0), (PAIR, 512, 600, 1544, 2048, 6),      # 512 wide: long enough to split its halves
    (LONE | dg.GEMM_FLAG_STAGE_K1, 256, 130, 264, 200, 0), (PAIR, 256, 1024, 512, 4096, 10), (LONE, 128, 256, 192, 4096, 5),
    (LONE, 512, 300, 512, 4096, 5), (PAIR, 512, 512, 768, 4096, 8), (LONE, 256, 5, 136, 8192, 0)])
def test_tiles(flags, tile, t, f, k, ctas, keep):
    info = run(t, f, k, torch.bfloat16, "silu", keep=keep, flags=flags, tile_n=tile, max_ctas=ctas)
    assert info.few_tiles == 0 and info.product.tile_n == tile and info.product.cta_group == (2 if flags & PAIR else 1)
    if ctas:
        assert info.product.stream_k_tiles > 0 or tile == 512


def test_values_that_are_not_finite_stay_in_their_row():
    for t in (5, 40):
        x, w = rows(t, 256, torch.bfloat16, 3), rows(128, 256, torch.bfloat16, 4, 0.1)
        out = torch.empty(t, 64, dtype=torch.bfloat16, device="cuda")
        with dg.GatedPlan(t, 64, 256) as p:
            clean = p.run(x, w, out).clone()
            x[1, 7], x[3, 255] = float("nan"), float("inf")
            w2 = w.clone()
            w2[5, 0] = float("nan")
            got = p.run(x, w2, out)
        keep = torch.ones(t, 64, dtype=torch.bool, device="cuda")
        keep[1] = keep[3] = False
        keep[:, 5] = False
        assert torch.equal(got[keep], clean[keep]) and got[1].isnan().all() and got[:, 5].isnan().all()


def test_far_arguments_of_the_activations():
    """Gates far out on both sides: no overflow inside, the limits at their ends."""
    k = 8
    x = torch.zeros(32, k, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([-1e4, -300.0, -90.0, -30.0, -12.0, -6.0, -1.0, -1e-3, 0.0, 1e-3, 1.0, 6.0, 12.0, 90.0, 300.0, 1e4] * 2, device="cuda")
    w = torch.zeros(16, k, dtype=torch.bfloat16, device="cuda")
    w[:8, 0] = 1.0          # gates: x itself
    w[8:, 1] = 1.0
    x[:, 1] = 1.0           # ups: one
    for act in ("silu", "gelu", "gelu_tanh"):
        for t in (16, 32):
            out = torch.empty(t, 8, dtype=torch.bfloat16, device="cuda")
            with dg.GatedPlan(t, 8, k, activation=act) as p:
                p.run(x[:t], w, out)
            want = act64(x[:t, :1].double(), act).expand(t, 8)
            # 2^-17 of the value and of the least that matters next to |g|: gelu's tails die out within fp32's range
            assert ((out.double() - want).abs() <= want.abs() * (half_step(torch.bfloat16) + 2.0 ** -17) + 1e-9).all(), (act, t)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dw_f32", [True, False])
@pytest.mark.parametrize("t,f,k,act", [(1, 8, 8, "silu"), (5, 64, 136, "gelu"), (96, 256, 520, "gelu_tanh"), (333, 264, 1001, "silu"), (1030, 512, 768, "gelu")])
def test_backward(t, f, k, act, dw_f32, kind):
    x, w, dh = rows(t, k, kind, 11, pad=8), rows(2 * f, k, kind, 12, k ** -0.5), rows(t, f, kind, 13)
    out = torch.empty(t, f, dtype=kind, device="cuda")
    gate_up = torch.empty(t, 2 * f, dtype=kind, device="cuda")
    with dg.GatedPlan(t, f, k, activation=act, dtype=CODE[kind], ldx=x.stride(0), ldw=w.stride(0), gradients=True,
                      dtype_dw=dg.GEMM_F32 if dw_f32 else None) as p:
        p.run(x, w, out, gate_up)
        dx, dw = p.backward(dh, x, w, gate_up)
        assert p.sync_status()[0] == dg.GEMM_OK
        assert dw.dtype == (torch.float32 if dw_f32 else kind)
        only_x, none = p.backward(dh, x, w, gate_up, need_dw=False)
        assert none is None and torch.equal(only_x, dx)
        both = gate_up.clone()
        dx2, dw2 = p.backward(dh, x, w, both, d_gate_up=both)         # the scratch over what was kept
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    g, u = (gate_up[:, i * f: (i + 1) * f].double().requires_grad_() for i in (0, 1))
    d = torch.cat(torch.autograd.grad(act64(g, act) * u, (g, u), dh.double()), 1)
    least = 2.0 ** -25 if kind == torch.float16 else 0.0
    # d_gate_up is rounded to 16 bits, after fp32 steps that are relative to |dh u| and |dh g|
    size = torch.cat((dh.double().abs() * u.detach().abs() * 1.2, dh.double().abs() * g.detach().abs()), 1)
    off = d.abs() * half_step(kind) + size * 2.0 ** -18 + least
    for got, want, bound, kd in (
            (dx, d @ w.double(), off @ w.double().abs() + (d.abs() @ w.double().abs()) * (2 * f * 2.0 ** -23), kind),
            (dw, d.T @ x.double(), off.T @ x.double().abs() + (d.abs().T @ x.double().abs()) * (t * 2.0 ** -23), dw.dtype)):
        bound = bound * 1.01 + want.abs() * half_step(kd) + least
        assert ((got.double() - want).abs() <= bound).all(), ((got.double() - want).abs() / bound).max().item()


def test_far_slopes():
    """Kept gates out to the ends of the types: slopes of 0 and 1, nothing of infinity times zero."""
    for kind, far in ((torch.bfloat16, 1e38), (torch.float16, 6e4)):
        t, f, k = 8, 8, 16
        gates = torch.tensor([-far, -far ** 0.5, -100.0, -50.0, 50.0, 100.0, far ** 0.5, far], device="cuda").to(kind)
        gate_up = torch.cat((gates.repeat(t, 1), torch.ones(t, f, dtype=kind, device="cuda")), 1)
        one, x, w = torch.ones(t, f, dtype=kind, device="cuda"), rows(t, k, kind, 5), rows(2 * f, k, kind, 6)
        for act in ("silu", "gelu", "gelu_tanh"):
            with dg.GatedPlan(t, f, k, activation=act, dtype=CODE[kind], gradients=True) as p:
                d = torch.empty(t, 2 * f, dtype=kind, device="cuda")
                p.backward(one, x, w, gate_up, d_gate_up=d)
                assert p.sync_status()[0] == dg.GEMM_OK
            # silu, whose tails are the longest: |silu'(g) - [g > 0]| <= (|g| + 1) e^-|g| and |silu(g) - max(g, 0)| <= |g| e^-|g|, at
            # |g| = 50 less than 51 * 1.93e-22 < 1e-20, far below the half step around 1 and 50
            assert ((d[:, :f].float() - (gates > 0).float()).abs() <= 1e-20).all(), act
            assert ((d[:, f:].float() - gates.float().clamp(min=0)).abs() <= 1e-20).all(), act


def test_backward_against_differences():
    t, f, k, kind = 24, 40, 72, torch.bfloat16
    x, w, dh = rows(t, k, kind, 21), rows(2 * f, k, kind, 22, 0.2), rows(t, f, kind, 23)
    out, gate_up = torch.empty(t, f, dtype=kind, device="cuda"), torch.empty(t, 2 * f, dtype=kind, device="cuda")
    for act in ("silu", "gelu", "gelu_tanh"):
        with dg.GatedPlan(t, f, k, activation=act, gradients=True, dtype_dw=dg.GEMM_F32) as p:
            p.run(x, w, out, gate_up)
            dx, dw = p.backward(dh, x, w, gate_up)
        def loss(a, b):
            both = a @ b.T
            return (act64(both[:, :f], act) * both[:, f:] * dh.double()).sum()
        step = 1e-5
        for got, at, other, first in ((dx, x, w, True), (dw, w, x, False)):
            v = torch.randn(at.shape, generator=torch.Generator(device="cuda").manual_seed(24), device="cuda").double()
            lo, hi = at.double() - step * v, at.double() + step * v
            o = other.double()
            slope = ((loss(hi, o) - loss(lo, o)) if first else (loss(o, hi) - loss(o, lo))) / (2 * step)
            # roundings of the kept sums and of d_gate_up, half a step each of bf16 and both times at most 1.2 of the magnitude,
            # and of the gradient itself; they are random in sign, so the worst case over the sum is generous
            assert abs((got.double() * v).sum() - slope) <= (got.double() * v).abs().sum() * half_step(kind) * 4


def test_no_tokens_and_refusals():
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), rows(128, 64, torch.bfloat16, 1)
    with dg.GatedPlan(0, 64, 64, gradients=True) as p:
        out = p.run(x, w, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
        dx, dw = p.backward(out, x, w, torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
        assert dx.shape == (0, 64) and (dw == 0).all()
    x, out, gu = rows(4, 64, torch.bfloat16, 2), torch.empty(4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    with dg.GatedPlan(4, 64, 64) as p:
        with pytest.raises(ValueError, match="without gradients"):
            p.backward(out, x, w, gu)
        with pytest.raises(ValueError, match="shape"):
            p.run(x[:3], w, out)
        with pytest.raises(TypeError):
            p.run(x.half(), w, out)
        with pytest.raises(ValueError, match="rows 72 apart"):
            p.run(rows(4, 64, torch.bfloat16, 2, pad=8), w, out)
        with pytest.raises(ValueError, match="CUDA device"):
            p.run(x.cpu(), w, out)


def test_streams_graphs_and_two_plans():
    kind = torch.bfloat16
    for t in (8, 200):
        f, k = 512, 1024
        x, w, dh = rows(t, k, kind, 31), rows(2 * f, k, kind, 32, 0.05), rows(t, f, kind, 33)
        outs = [torch.empty(t, f, dtype=kind, device="cuda") for _ in range(2)]
        gate_up = torch.empty(t, 2 * f, dtype=kind, device="cuda")
        plans = [dg.GatedPlan(t, f, k, gradients=True) for _ in range(2)]
        want = plans[0].run(x, w, outs[0], gate_up).clone()
        want_dx, want_dw = (v.clone() for v in plans[0].backward(dh, x, w, gate_up))
        # two plans at once on two streams
        sides = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(8):
            for p, s, o in zip(plans, sides, outs):
                p.run(x, w, o, stream=s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plans[0].run(x, w, outs[0], gate_up)
            dx, dw = plans[0].backward(dh, x, w, gate_up)
        x2 = rows(t, k, kind, 34)
        keep = x.clone()
        x.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        assert not torch.equal(outs[0], want)
        check_forward(x2, w, "silu", outs[0], gate_up)
        x.copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
        for p in plans:
            assert p.sync_status()[0] == dg.GEMM_OK
            p.close()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,f,k", [(100, 9736, 128), (128, 9728, 72), (96, 19472, 64), (3, 19464, 72)])
def test_few_tokens_of_wide_layers(t, f, k, kind):
    """97 to 128 tokens of layers wide enough for the pipeline, and columns that one wave of CTAs does not hold."""
    assert run(t, f, k, kind, "silu", keep=t % 2 == 0).few_tiles == 0


def test_backward_many_turns():
    """The pass over memory takes its grid two and a half times over H."""
    test_backward(3000, 2048, 64, "gelu", True, torch.bfloat16)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dw_f32", [True, False])
@pytest.mark.parametrize("t,f,act", [(2304, 1152, "silu"), (2300, 1144, "gelu_tanh")])
def test_backward_wide_tiles(t, f, act, dw_f32, kind):
    """Both products in 512-wide tiles, with tokens and features of whole groups of 64 and not."""
    k = 4096
    with dg.GatedPlan(t, f, k, dtype=CODE[kind], gradients=True, dtype_dw=dg.GEMM_F32 if dw_f32 else None) as p:
        assert p.info.dx.tile_n == 512 and p.info.dw.tile_n == 512
    test_backward(t, f, k, act, dw_f32, kind)


def test_backward_of_few_tokens_takes_no_wide_tiles():
    with dg.GatedPlan(64, 8192, 32768, gradients=True) as p:
        assert p.info.dx.tile_n <= 256 and p.info.dw.tile_n <= 256


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,f,k,split", [(130, 512, 28672, True), (200, 1000, 16392, True), (260, 136, 12288, True), (130, 1024, 6144, False)])
def test_few_tiles_of_a_long_k_share_it(t, f, k, split, kind):
    info = run(t, f, k, kind, "silu", keep=t != 200)
    assert info.few_tiles == 0 and (info.product.stream_k_tiles > 0) == split
