"""GPU: the residual's addition and its RMS norm against a 64-bit form: widths off every boundary, padded and in-place rows, both
8-bit outputs and the products that read them, values that are not finite, streams and graphs; and the backward pass against the
formula and against differences."""
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg
from dense_gemm_blackwell_gb300 import inputs  # noqa: F401  (scale tiles' layout is described there)

pytestmark = pytest.mark.gpu

BLOCK, MX = dg.GEMM_SCALE_BLOCK_1x128_128x128, dg.GEMM_SCALE_MX_E8M0_32
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
# fp32 steps on the way to a value: the sum of squares (its relative error is halved by the root), rsqrt, two products and a
# scale; 64 of them cover the longest sum of a thread and the joins
FP32 = 64 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def rows(t, n, kind, seed, scale=1.0, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ld = -(-n // 8) * 8 + pad
    return (torch.randn(t, ld, generator=gen, device="cuda") * scale).to(kind)[:, :n]


def weights(n, kind, seed=9):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(n, generator=gen, device="cuda")).to(kind)


def exact(h, weight):
    h = h.double()
    y = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    return y if weight is None else y * weight.double()


def half_step(kind):
    return torch.finfo(kind).eps / 2


def near(got, want, kind):
    least = 2.0 ** -25 if kind == torch.float16 else 0.0       # half the smallest step of f16
    err = (got.double() - want).abs()
    assert (err <= want.abs() * (half_step(kind) + FP32) + least).all(), err.max().item()


def untile(bytes_, t, n):
    """Scale exponents [t, ceil(n / 32)] out of the tiles, and the bytes past the matrix."""
    kb = -(-n // 32)
    wide = -(-kb // 4)
    r = torch.arange(t, device="cuda")[:, None]
    q = torch.arange(kb, device="cuda")[None, :]
    at = (r // 128 * wide + q // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + q % 4
    rest = torch.ones(bytes_.numel(), dtype=torch.bool, device="cuda")
    rest[at.flatten()] = False
    return bytes_[at].int(), bytes_[rest]


SIZES = [(1, 8), (1, 1), (3, 7), (5, 129), (130, 256), (1, 4096), (257, 2893), (33, 8192), (7, 8200), (2, 16384), (3, 32768), (700, 264),
         (1000, 1000)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", SIZES)
def test_forward(t, n, kind):
    x, res, w = rows(t, n, kind, 1, pad=16), rows(t, n, kind, 2, 3.0), weights(n, kind)
    y, scales, h = dg.add_rms_norm(x, w, residual=res, eps=EPS)
    assert scales is None
    assert torch.equal(h, (x.float() + res.float()).to(kind))
    near(y, exact(h, w), kind)
    y2, _, none = dg.add_rms_norm(x, eps=EPS)
    assert none is None
    near(y2, exact(x, None), kind)


def check_codes(codes, scale, want):
    """Codes times scales: half a step of the code, of the least step under 2^-6, and fp32 next to nothing."""
    got = codes.double() * scale
    bound = (want.abs() * 2.0 ** -4).maximum(scale * 2.0 ** -10) * (1 + 2.0 ** -18) + want.abs() * FP32
    assert ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", SIZES)
def test_block_scales(t, n, kind):
    x, res, w = rows(t, n, kind, 3), rows(t, n, kind, 4, 3.0, pad=8), weights(n, kind)
    codes, scales, h = dg.add_rms_norm(x, w, residual=res, eps=EPS, scale_mode=BLOCK)
    assert codes.dtype == E4M3 and torch.equal(h, (x.float() + res.float()).to(kind))
    want = exact(h, w)
    top = torch.nn.functional.pad(want.abs(), (0, -n % 128)).unflatten(1, (-1, 128)).amax(2)
    assert ((scales.double() - top / 448).abs() <= top / 448 * FP32).all()
    check_codes(codes, scales.double().repeat_interleave(128, 1)[:, :n], want)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", SIZES)
def test_tiled_scales(t, n, kind):
    x, w = rows(t, n, kind, 5), weights(n, kind)
    room = torch.full((-(-t // 128) * -(-n // 128) * 512,), 0xAA, dtype=torch.uint8, device="cuda")
    codes, scales, h = dg.add_rms_norm(x, w, eps=EPS, scale_mode=MX, scales=room)
    assert h is None and scales is room
    e, rest = untile(scales, t, n)
    assert (rest == 0).all()
    want = exact(x, w)
    top = torch.nn.functional.pad(want.abs(), (0, -n % 32)).unflatten(1, (-1, 32)).amax(2)
    s = torch.exp2(e.double() - 127)
    assert (top <= 448 * s * (1 + FP32)).all() and ((top > 224 * s * (1 - FP32)) | (e == 1)).all()
    check_codes(codes, s.repeat_interleave(32, 1)[:, :n], want)


def test_rows_of_zeros_and_tiny_rows():
    x = torch.zeros(5, 300, dtype=torch.bfloat16, device="cuda")
    x = torch.nn.functional.pad(x, (0, 4))[:, :300]
    x[1, 5] = 2.0 ** -60
    x[3, 299] = -1.0
    for mode, least in ((BLOCK, 2.0 ** -100), (MX, None)):
        codes, scales, _ = dg.add_rms_norm(x, eps=0.0 if mode == MX else 1e-6, scale_mode=mode)
        got = codes.float()
        if mode == BLOCK:
            assert (got[0] == 0).all() and (scales[0] == least).all() and (scales[4] == least).all()
            assert got[1].abs().max() > 0 and (got[1] != 0).sum() == 1
        else:       # 0 / sqrt(0): NaN rows stay NaN, and the others are untouched
            assert got[0].isnan().all() and got[2].isnan().all() and got[3, 299] < 0 and (got[3, :299] == 0).all()


@pytest.mark.parametrize("mode", [dg.GEMM_SCALE_NONE, BLOCK, MX])
def test_values_that_are_not_finite_stay_in_their_row(mode):
    x = rows(6, 1000, torch.bfloat16, 6)
    x[1, 17] = float("nan")
    x[4, 999] = float("inf")
    w = weights(1000, torch.bfloat16)
    got = dg.add_rms_norm(x, w, eps=EPS, scale_mode=mode)[0].float()
    assert got[1].isnan().all()
    assert got[4, 999].isnan() and (got[4, :999] == 0).all()
    clean = torch.tensor([0, 2, 3, 5], device="cuda")
    alone = dg.add_rms_norm(x[clean], w, eps=EPS, scale_mode=mode)[0].float()
    assert torch.equal(got[clean], alone)


def test_infinite_sums():
    big = torch.full((1, 64), 60000.0, dtype=torch.float16, device="cuda")
    y, _, h = dg.add_rms_norm(big, residual=big)
    assert h.isinf().all() and y.isnan().all()


def test_in_place_and_what_lies_around():
    t, n, kind = 37, 1234, torch.bfloat16
    x, w = rows(t, n, kind, 7), weights(n, kind)
    want_y, _, want_h = dg.add_rms_norm(x, w, residual=rows(t, n, kind, 8))
    store = torch.full((t + 2, 1248), 7.0, dtype=kind, device="cuda")
    res = store[1: t + 1, :n]
    res.copy_(rows(t, n, kind, 8))
    out = torch.full((t + 2, 1240), 5.0, dtype=kind, device="cuda")
    y, _, h = dg.add_rms_norm(x, w, residual=res, sum_out=res, out=out[1: t + 1, :n])
    assert torch.equal(h, want_h) and torch.equal(y, want_y)
    assert (store[0] == 7).all() and (store[-1] == 7).all() and (store[:, n:] == 7).all()
    assert (out[0] == 5).all() and (out[-1] == 5).all() and (out[:, n:] == 5).all()
    # out over x, the sum over the residual
    x2, res2 = x.clone(), rows(t, n, kind, 8).clone()
    res2 = torch.nn.functional.pad(res2, (0, 6))[:, :n]
    x2 = torch.nn.functional.pad(x2, (0, 6))[:, :n]
    y, _, h = dg.add_rms_norm(x2, w, residual=res2, sum_out=res2, out=x2)
    assert torch.equal(x2, want_y) and torch.equal(res2, want_h)
    codes = torch.zeros(t, 1264, dtype=torch.uint8, device="cuda").fill_(0x55)
    scales = torch.full((t, 12), 3.0, device="cuda")
    dg.add_rms_norm(x, w, out=codes.view(E4M3)[:, :n], scale_mode=BLOCK, scales=scales[:, :10])
    assert (codes[:, n:] == 0x55).all() and (scales[:, 10:] == 3).all()


def test_no_tokens_and_refusals():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, _, h = dg.add_rms_norm(x, residual=x)
    assert y.shape == h.shape == (0, 64)
    dh, dw = dg.add_rms_norm_backward(x, x, weights(64, torch.bfloat16))
    assert dh.shape == (0, 64) and (dw == 0).all()
    x = rows(4, 64, torch.bfloat16, 1)
    with pytest.raises(TypeError):
        dg.add_rms_norm(x.float())
    with pytest.raises(TypeError):
        dg.add_rms_norm(x, residual=x.half())
    with pytest.raises(ValueError, match="rows overlap"):
        dg.add_rms_norm(x, out=torch.zeros(64, dtype=torch.bfloat16, device="cuda").expand(4, 64))
    with pytest.raises(ValueError, match="contiguous"):
        dg.add_rms_norm(rows(64, 4, torch.bfloat16, 1).T)
    with pytest.raises(ValueError, match="shape"):
        dg.add_rms_norm(x, residual=rows(4, 72, torch.bfloat16, 1))
    with pytest.raises(ValueError, match="scales"):
        dg.add_rms_norm(x, scales=torch.zeros(4, 1, device="cuda"))
    with pytest.raises(dg.GemmError):
        dg.add_rms_norm(torch.zeros(4, 65, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="CUDA device"):
        dg.add_rms_norm(x, residual=x.cpu())


@pytest.mark.parametrize("mode", [BLOCK, MX])
def test_into_the_product(mode):
    """The codes and scales are the product's A: its result is that of the decoded rows."""
    t, n, k = 200, 384, 640
    x, w = rows(t, k, torch.bfloat16, 11), weights(k, torch.bfloat16)
    codes, scales, _ = dg.add_rms_norm(x, w, scale_mode=mode)
    b = (torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(12), device="cuda")).to(E4M3)
    if mode == BLOCK:
        sb = torch.rand(-(-n // 128), -(-k // 128), generator=torch.Generator(device="cuda").manual_seed(13), device="cuda") + 0.5
        d = dg.matmul(codes, b, scale_a=scales, scale_b=sb)
        a64 = codes.double() * scales.double().repeat_interleave(128, 1)[:, :k]
        b64 = b.double() * sb.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    else:
        sfb = torch.full((-(-n // 128) * -(-k // 128) * 512,), 127, dtype=torch.uint8, device="cuda")
        d = torch.empty(t, n, device="cuda")
        with dg.Plan(dg.make_desc(t, n, k, dtype_a=dg.GEMM_E4M3, scale_mode=MX)) as plan:
            plan.run_mx(codes, b, d, scales, sfb)
            assert plan.sync_status()[0] == dg.GEMM_OK
        a64 = codes.double() * torch.exp2(untile(scales, t, k)[0].double() - 127).repeat_interleave(32, 1)[:, :k]
        b64 = b.double()
    want = a64 @ b64.T
    size = a64.abs() @ b64.abs().T
    assert ((d.double() - want).abs() <= size * k * 2.0 ** -23).all()


# ---------------------------------------------------------------- backward

def exact_backward(dy, h, weight, dsum):
    h = h.double().requires_grad_()
    w = None if weight is None else weight.double().requires_grad_()
    y = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
    if w is not None:
        y = y * w
    found = torch.autograd.grad(y, [h] + ([] if w is None else [w]), dy.double())
    return found[0] + (0 if dsum is None else dsum.double()), None if w is None else found[1]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", SIZES + [(5000, 320)])
def test_backward(t, n, kind):
    h, dy, dsum, w = rows(t, n, kind, 21, 2.0), rows(t, n, kind, 22, pad=8), rows(t, n, kind, 23), weights(n, kind)
    for weight, along in ((w, dsum), (None, None), (w, None)):
        dh, dw = dg.add_rms_norm_backward(dy, h, weight, d_sum=along, eps=EPS)
        want, want_w = exact_backward(dy, h, weight, along)
        r = 1 / (h.double().pow(2).mean(1, keepdim=True) + EPS).sqrt()
        u = h.double() * r
        gw = (dy if weight is None else dy.double() * weight.double()).double()
        size = (r * gw).abs() + (r * u).abs() * (gw * u).abs().mean(1, keepdim=True) + (0 if along is None else along.double().abs())
        least = 2.0 ** -25 if kind == torch.float16 else 0.0
        assert ((dh.double() - want).abs() <= want.abs() * half_step(kind) + size * FP32 + least).all()
        assert (dw is None) == (weight is None)
        if dw is not None:
            # a sum of t terms in a fixed order: at most t steps of fp32 beside each term's own
            assert ((dw.double() - want_w).abs() <= (dy.double() * u).abs().sum(0) * ((t + 64) * 2.0 ** -24)).all()
            again = dg.add_rms_norm_backward(dy, h, weight, d_sum=along, eps=EPS)[1]
            assert torch.equal(dw, again)


def test_backward_against_differences():
    t, n = 9, 72
    kind = torch.bfloat16
    h, dy, w = rows(t, n, kind, 31, 2.0), rows(t, n, kind, 32), weights(n, kind)
    dh, dw = dg.add_rms_norm_backward(dy, h, w, eps=EPS)
    f = lambda a, b: (exact(a, b) * dy.double()).sum()  # noqa: E731
    step = 1e-5
    v = torch.randn(t, n, generator=torch.Generator(device="cuda").manual_seed(33), device="cuda").double()
    slope = (f(h.double() + step * v, w.double()) - f(h.double() - step * v, w.double())) / (2 * step)
    assert abs((dh.double() * v).sum() - slope) <= (dh.double() * v).abs().sum() * half_step(kind) * 2 + 1e-6
    vw = v[0]
    slope = (f(h.double(), w.double() + step * vw) - f(h.double(), w.double() - step * vw)) / (2 * step)
    assert abs((dw.double() * vw).sum() - slope) <= (dw.double() * vw).abs().sum() * 1e-5 + 1e-6


def test_backward_of_tiny_rows_without_eps():
    """r^3 is past fp32's range where r and the gradients are not."""
    t, n, kind = 5, 200, torch.bfloat16
    h, dy, w = rows(t, n, kind, 34) * 2.0 ** -50, rows(t, n, kind, 35), weights(n, kind)
    dh, dw = dg.add_rms_norm_backward(dy, h, w, eps=0.0)
    want, want_w = dg.add_rms_norm_backward(dy, h * 2.0 ** 50, w, eps=0.0)
    assert want.isfinite().all() and torch.equal(dh * 2.0 ** -50, want) and torch.equal(dw, want_w)


@pytest.mark.parametrize("n", [1000, 12000])
def test_backward_in_place(n):
    t, kind = 40, torch.bfloat16
    h, dy, dsum, w = rows(t, n, kind, 41, 2.0), rows(t, n, kind, 42), rows(t, n, kind, 43), weights(n, kind)
    want, want_w = dg.add_rms_norm_backward(dy, h, w, d_sum=dsum)
    for over in ("dy", "dsum", "h"):
        c = dict(dy=dy.clone(), dsum=dsum.clone(), h=h.clone())
        c = {k: torch.nn.functional.pad(v, (0, -n % 8))[:, :n] for k, v in c.items()}
        dh, dw = dg.add_rms_norm_backward(c["dy"], c["h"], w, d_sum=c["dsum"], out=c[over])
        assert torch.equal(dh, want) and torch.equal(dw, want_w)


def test_streams_and_graphs():
    t, n, kind = 64, 4096, torch.bfloat16
    x, res, w = rows(t, n, kind, 51), rows(t, n, kind, 52), weights(n, kind)
    want = dg.add_rms_norm(x, w, residual=res, scale_mode=MX)
    want_g = dg.add_rms_norm_backward(x, res, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = dg.add_rms_norm(x, w, residual=res, scale_mode=MX, stream=side.cuda_stream)      # not behind the default stream
    got_g = dg.add_rms_norm_backward(x, res, w, stream=side.cuda_stream)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.uint8) if a.dtype == E4M3 else a, b.view(torch.uint8) if b.dtype == E4M3 else b)  # noqa: E731
    assert all(same(a, b) for a, b in zip(want, got)) and all(same(a, b) for a, b in zip(want_g, got_g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dg.add_rms_norm(x, w, residual=res, scale_mode=MX)
        got_g = dg.add_rms_norm_backward(x, res, w)
    x2 = rows(t, n, kind, 53)
    want, want_g = dg.add_rms_norm(x2, w, residual=res, scale_mode=MX), dg.add_rms_norm_backward(x2, res, w)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(want, got)) and all(same(a, b) for a, b in zip(want_g, got_g))


# ---------------------------------------------------------------- blocks that take row after row

# With 152 SMs: 3 turns of one row a block and 6 warps a row, 4 of 16 warps, 2 of four rows a block, 5 of four vectors a thread
MANY = [(2500, 2893), (1500, 8192), (9000, 264), (700, 20000)]


def check_scaled(mode, codes, scales, want):
    t, n = want.shape
    size = 128 if mode == BLOCK else 32
    top = torch.nn.functional.pad(want.abs(), (0, -n % size)).unflatten(1, (-1, size)).amax(2)
    if mode == BLOCK:
        s = scales.double()
        assert ((s - top / 448).abs() <= top / 448 * FP32).all()
    else:
        e, rest = untile(scales, t, n)
        assert (rest == 0).all()
        s = torch.exp2(e.double() - 127)
        assert (top <= 448 * s * (1 + FP32)).all() and ((top > 224 * s * (1 - FP32)) | (e == 1)).all()
    check_codes(codes, s.repeat_interleave(size, 1)[:, :n], want)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mode", [dg.GEMM_SCALE_NONE, BLOCK, MX])
@pytest.mark.parametrize("t,n", MANY)
def test_many_turns(t, n, mode, kind):
    w = weights(n, kind)
    for res, weight in ((True, w), (True, None), (False, w)):
        x, r = rows(t, n, kind, 61, pad=8), rows(t, n, kind, 62, 3.0) if res else None
        room = torch.full((-(-t // 128) * -(-n // 128) * 512,), 0xAA, dtype=torch.uint8, device="cuda") if mode == MX else None
        y, scales, h = dg.add_rms_norm(x, weight, residual=r, eps=EPS, scale_mode=mode, scales=room)
        if res:
            assert torch.equal(h, (x.float() + r.float()).to(kind))
        want = exact(h if res else x, weight)
        if mode == dg.GEMM_SCALE_NONE:
            near(y, want, kind)
        else:
            check_scaled(mode, y, scales, want)
        # the sum over the residual (or x); a 16-bit output over x: every turn reads its rows before it writes them
        x2, r2 = x.clone(memory_format=torch.preserve_format), r.clone(memory_format=torch.preserve_format) if res else None
        over = torch.nn.functional.pad(x2, (0, -n % 8))[:, :n]
        sum2 = torch.nn.functional.pad(r2, (0, -n % 8))[:, :n] if res else None
        for _ in range(2):
            over.copy_(x)
            if res:
                sum2.copy_(r)
            y2, scales2, h2 = dg.add_rms_norm(over, weight, residual=sum2, eps=EPS, scale_mode=mode, out=over if mode == dg.GEMM_SCALE_NONE else None,
                                              sum_out=sum2)
            assert torch.equal(y2.view(torch.uint8) if mode else y2, y.view(torch.uint8) if mode else y)
            assert scales is None or torch.equal(scales2, scales)
            assert not res or torch.equal(h2, h)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", SIZES)
def test_tiled_scales_of_a_sum(t, n, kind):
    x, res, w = rows(t, n, kind, 63), rows(t, n, kind, 64, 3.0, pad=8), weights(n, kind)
    codes, scales, h = dg.add_rms_norm(x, w, residual=res, eps=EPS, scale_mode=MX)
    assert torch.equal(h, (x.float() + res.float()).to(kind))
    check_scaled(MX, codes, scales, exact(h, w))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("t,n", [(3000, 4096), (2500, 2893), (1200, 9000), (800, 20000), (9000, 264)])
def test_backward_many_turns(t, n, kind):
    test_backward(t, n, kind)
    h, dy, dsum, w = rows(t, n, kind, 71, 2.0), rows(t, n, kind, 72), rows(t, n, kind, 73), weights(n, kind)
    want, want_w = dg.add_rms_norm_backward(dy, h, w, d_sum=dsum)
    for over in ("dy", "dsum", "h"):
        c = {k: torch.nn.functional.pad(v, (0, -n % 8))[:, :n] for k, v in dict(dy=dy.clone(), dsum=dsum.clone(), h=h.clone()).items()}
        dh, dw = dg.add_rms_norm_backward(c["dy"], c["h"], w, d_sum=c["dsum"], out=c[over])
        assert torch.equal(dh, want) and torch.equal(dw, want_w)


@pytest.mark.parametrize("mode", [BLOCK, MX])
def test_a_weight_that_is_not_a_number_stays_in_its_column(mode):
    """Its code is NaN in every row; the block's scale and other codes are those without it."""
    x, w = rows(40, 1000, torch.bfloat16, 81), weights(1000, torch.bfloat16)
    w[333] = 0
    want, want_scales, _ = dg.add_rms_norm(x, w, eps=EPS, scale_mode=mode)
    w[333] = float("nan")
    got, scales, _ = dg.add_rms_norm(x, w, eps=EPS, scale_mode=mode)
    others = torch.arange(1000, device="cuda") != 333
    assert got.float()[:, 333].isnan().all() and torch.equal(scales, want_scales)
    assert torch.equal(got.view(torch.uint8)[:, others], want.view(torch.uint8)[:, others])
