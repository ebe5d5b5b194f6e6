"""GPU: products of a few tokens with 4-bit weights against a 64-bit form: every group width and token count, odd sizes, padded
rows, zero points, gated pairs, values that are not finite, streams and graphs."""
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def make(t, n, k, group, kind, zeros, seed=1, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    groups = -(-k // group)
    x = torch.randn(t, -(-k // 8) * 8 + pad, generator=gen, device="cuda").to(kind)[:, :k]
    codes = torch.randint(0, 256, (n, -(-k // 32) * 16 + 2 * pad), generator=gen, device="cuda").to(torch.uint8)[:, : k // 2]
    scales = ((0.5 + torch.rand(n, groups + pad, generator=gen, device="cuda")) * 0.25 * k ** -0.5).to(kind)[:, :groups]
    z = torch.randint(0, 16, (n, groups + pad), generator=gen, device="cuda").to(torch.uint8)[:, :groups] if zeros else None
    return x, codes, scales, z


def decode(codes, scales, zeros, k, group):
    w = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double()
    at = torch.arange(k, device="cuda") // group
    return (w - (8.0 if zeros is None else zeros.double()[:, at])) * scales.double()[:, at]


def act64(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")


def check(y, x, codes, scales, zeros, group, act=None):
    k, kind = x.shape[1], x.dtype
    w = decode(codes, scales, zeros, k, group)
    p = x.double() @ w.T
    err = (x.double().abs() @ w.abs().T) * (min(k, 4096) * 2.0 ** -23)        # fp32 sums, at most a step an element
    half = torch.finfo(kind).eps / 2
    least = 2.0 ** -25 if kind == torch.float16 else 0.0
    if act is None:
        want, bound = p, err
    else:
        n = p.shape[1] // 2
        g, u, a = p[:, :n], p[:, n:], act64(p[:, :n], act)
        want, bound = a * u, 1.13 * err[:, :n] * (u.abs() + err[:, n:]) + a.abs() * err[:, n:] + g.abs() * u.abs() * 2.0 ** -19
    bound = bound + (want.abs() + bound) * half + least
    assert ((y.double() - want).abs() <= bound).all(), ((y.double() - want).abs() / bound).max().item()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 160, 192, 256, 512])
@pytest.mark.parametrize("t,n,k", [(1, 4096, 4096), (1, 1, 2), (3, 33, 130), (8, 100, 1024), (9, 47, 2050), (13, 1543, 5130), (16, 640, 768)])
def test_product(t, n, k, group, kind):
    zeros = (n + group // 32) % 2 == 0
    x, codes, scales, z = make(t, n, k, group, kind, zeros, pad=8 * (t % 2))
    store = torch.full((t + 1, n + 3), 7.0, dtype=kind, device="cuda")
    y = dg.int4_matmul(x, codes, scales, group=group, zeros=z, out=store[:t, :n])
    check(y, x, codes, scales, z, group)
    assert (store[t:] == 7).all() and (store[:, n:] == 7).all()
    assert torch.equal(dg.int4_matmul(x, codes, scales, group=group, zeros=z), y)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t,n,k,group", [(1, 2048, 4096, 128), (5, 17, 66, 32), (8, 1000, 2048, 64), (12, 333, 4100, 128), (16, 48, 12288, 256)])
def test_gated(t, n, k, group, act, kind):
    x, codes, scales, z = make(t, 2 * n, k, group, kind, n % 2 == 1, seed=2)
    y = dg.int4_matmul(x, codes, scales, group=group, zeros=z, activation=act)
    assert y.shape == (t, n)
    check(y, x, codes, scales, z, group, act)


@pytest.mark.parametrize("t,n,k,group,act", [
    (1, 40000, 512, 128, None), (5, 20011, 1536, 64, "silu"), (3, 9000, 700, 32, None), (16, 8200, 28672, 128, None), (12, 4100, 28672, 128, "gelu"),
    (8, 16411, 4096, 128, "silu"), (11, 30000, 2560, 96, None)])
def test_many_tiles_a_block(t, n, k, group, act):
    """Tiles inside a warp's run, tiles that several warps share, and, of a K that a cluster shares, several joins."""
    x, codes, scales, z = make(t, n if act is None else 2 * n, k, group, torch.bfloat16 if t % 2 else torch.float16, True, seed=9)
    y = dg.int4_matmul(x, codes, scales, group=group, zeros=z, activation=act)
    for at in range(0, n, 4096):        # the 64-bit form of some rows at a time
        pick = torch.arange(at, min(n, at + 4096), device="cuda")
        rows = pick if act is None else torch.cat((pick, pick + n))
        check(y[:, pick], x, codes[rows], scales[rows], z[rows], group, act)
    assert torch.equal(dg.int4_matmul(x, codes, scales, group=group, zeros=z, activation=act), y)


@pytest.mark.parametrize("t,n,k,group", [(16, 70, 28672, 128), (16, 33, 45056, 32), (8, 40, 49154, 64), (8, 33, 94208, 32), (1, 17, 94208, 256)])
def test_long_k(t, n, k, group):
    """X of a block takes a cluster of eight's shared memory, at last that of whole SMs."""
    x, codes, scales, z = make(t, n, k, group, torch.bfloat16, True, seed=8)
    check(dg.int4_matmul(x, codes, scales, group=group, zeros=z), x, codes, scales, z, group)


def test_too_long_k_is_refused():
    for t, k in ((1, 131072), (9, 65536)):
        x, codes, scales, z = make(t, 8, k, 128, torch.bfloat16, False)
        with pytest.raises(dg.GemmError):
            dg.int4_matmul(x, codes, scales)


def test_every_code_is_exact():
    """One element of x at a time picks a column of W out: scale times (code - zero), rounded once."""
    k, n = 64, 256
    for kind in (torch.bfloat16, torch.float16):
        codes = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, k // 2)
        zeros = (torch.arange(n, device="cuda") % 128).to(torch.uint8)[:, None].repeat(1, 2)
        scales = torch.full((n, 2), 0.5, dtype=kind, device="cuda")
        x = torch.zeros(16, k, dtype=kind, device="cuda")
        at = torch.arange(16, device="cuda") * 4 + torch.arange(16, device="cuda") % 4
        x[torch.arange(16, device="cuda"), at] = 1.0
        y = dg.int4_matmul(x, codes, scales, group=32, zeros=zeros)
        assert torch.equal(y.double(), decode(codes, scales, zeros, k, 32)[:, at].T)


def test_values_that_are_not_finite_stay_where_they_are():
    for t in (4, 11):
        x, codes, scales, z = make(t, 70, 1030, 32, torch.bfloat16, True, seed=3)
        clean = dg.int4_matmul(x, codes, scales, group=32, zeros=z)
        x, scales = x.clone(), scales.clone()
        x = torch.nn.functional.pad(x, (0, 2))[:, :1030]
        x[1, 1029], x[3, 0] = float("nan"), float("inf")
        scales[5, 32], scales[40, 0] = float("nan"), float("inf")
        y = dg.int4_matmul(x, codes, scales, group=32, zeros=z)
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[1] = keep[3] = False
        keep[:, 5] = keep[:, 40] = False
        assert torch.equal(y[keep], clean[keep]) and y[1].isnan().all() and y[:, 5].isnan().all()
        assert not y[:, 40].isfinite().any()


def test_padding_is_not_read_into_the_sums():
    x, codes, scales, z = make(7, 50, 1100, 128, torch.bfloat16, True, seed=4)
    want = dg.int4_matmul(x, codes, scales, zeros=z)
    wide = torch.full((7, 1104 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :1100] = x
    assert torch.equal(dg.int4_matmul(wide[:, :1100], codes, scales, zeros=z), want)


def test_no_tokens_and_refusals():
    x, codes, scales, z = make(4, 32, 64, 32, torch.bfloat16, True)
    assert dg.int4_matmul(x[:0], codes, scales, group=32, zeros=z).shape == (0, 32)
    with pytest.raises(TypeError):
        dg.int4_matmul(x, codes, scales.half(), group=32)
    with pytest.raises(TypeError):
        dg.int4_matmul(x, codes.int(), scales, group=32)
    with pytest.raises(ValueError, match="shape"):
        dg.int4_matmul(x, codes, scales, group=64)
    with pytest.raises(ValueError, match="activation"):
        dg.int4_matmul(x, codes, scales, group=32, activation="relu")
    with pytest.raises(ValueError, match="even"):
        dg.int4_matmul(x[:, :63], codes, scales, group=32)
    with pytest.raises(ValueError, match="CUDA device"):
        dg.int4_matmul(x, codes.cpu(), scales, group=32)
    with pytest.raises(dg.GemmError):
        many = torch.zeros(17, 64, dtype=torch.bfloat16, device="cuda")
        dg.int4_matmul(many, codes, scales, group=32)
    with pytest.raises(dg.GemmError):
        x3, c3, s3, _ = make(4, 32, 96, 48, torch.bfloat16, False)
        dg.int4_matmul(x3, c3, s3, group=48)


def test_quantized_weights():
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(96, 1000, generator=gen, device="cuda").to(torch.bfloat16)
    x = torch.randn(3, 1000, generator=gen, device="cuda").to(torch.bfloat16)
    for symmetric in (True, False):
        codes, scales, zeros = dg.int4_quantize(w, 64, symmetric=symmetric)
        y = dg.int4_matmul(x, codes, scales, group=64, zeros=zeros)
        check(y, x, codes, scales, zeros, 64)
        # and near the product with w itself: every weight within a step (and a half) of its group's scale
        off = x.double().abs() @ (scales.double().repeat_interleave(64, 1)[:, :1000] * 1.1).T
        assert ((y.double() - x.double() @ w.double().T).abs() <= off).all()


def test_streams_and_graphs():
    x, codes, scales, z = make(6, 2048, 2048, 128, torch.bfloat16, True, seed=6)
    want = dg.int4_matmul(x, codes, scales, zeros=z, activation="silu")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = dg.int4_matmul(x, codes, scales, zeros=z, activation="silu", stream=side.cuda_stream)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dg.int4_matmul(x, codes, scales, zeros=z, activation="silu")
    x.copy_(make(6, 2048, 2048, 128, torch.bfloat16, True, seed=7)[0])
    graph.replay()
    torch.cuda.synchronize()
    check(got, x, codes, scales, z, 128, "silu")
