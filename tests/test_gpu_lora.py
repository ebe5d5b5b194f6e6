"""GPU: a shared projection with low-rank adapters, against a plain 64-bit form.

Exact cases: inputs from small integers and scales that are powers of two, so that every sum is an integer or a half
below 2^24 and every T (at most 8 significant bits) is its own 16-bit rounding; Y must be the 64-bit result rounded once,
bit for bit, whatever kernel, tile or split computed it.

Random cases: with S = sum |x||w| + s sum_r (sum_k |x||a|) |b| the sum of all magnitudes an element adds up,
  |Y - Y64| <= (k / 8 + 16) 2^-23 S        fp32 accumulation, a tensor-core step (16 products) adding at most two units
                                           in the last place of a running sum that is at most S, for X W^T and T alike
             + u D                         T rounded to the input type (u = 2^-8 bf16, 2^-11 f16), D = s sum_r |T||b|;
                                           for fp32 outputs T is two terms: u^2
             + u_out (|Y64| + the above)   the output's rounding.
"""
import threading

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: dg.GEMM_BF16, torch.float16: dg.GEMM_F16, torch.float32: dg.GEMM_F32}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def padded(t):
    """The same matrix with rows 16 bytes apart or more, NaN behind them."""
    ld = -(-t.shape[-1] // 8) * 8 + 8
    full = torch.full(t.shape[:-1] + (ld,), NAN, dtype=t.dtype, device=t.device)
    full[..., : t.shape[-1]] = t
    return full[..., : t.shape[-1]]


def ints(gen, *shape, lo=-1, hi=1, density=1.0):
    v = torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").double()
    return v * (torch.rand(shape, generator=gen, device="cuda") < density) if density < 1 else v


def ids_for(kind, tokens, adapters, gen):
    if kind == "none":
        return torch.full((tokens,), -1, device="cuda", dtype=torch.int32)
    if kind == "one":
        return torch.full((tokens,), adapters - 1, device="cuda", dtype=torch.int32)
    if kind == "runs":          # prompts: long runs, one of them without an adapter
        return (torch.arange(tokens, device="cuda") * 5 // max(tokens, 1) % (adapters + 1) - 1).to(torch.int32)
    r = torch.randint(-1, adapters, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    if kind == "wild":          # numbers that name no adapter
        r[::3] = -7
        r[1::5] = adapters
        r[2::7] = 2 ** 31 - 1
    return r


def plain(x, w, a, b, adapter, scale):
    """Y and T's contribution in 64 bits."""
    y = x @ w.T
    for i in range(a.shape[0]):
        rows = (adapter == i).nonzero().flatten()
        if len(rows):
            y[rows] += scale[i] * ((x[rows] @ a[i].T) @ b[i].T)
    return y


def make_exact(tokens, n, k, rank, adapters, kind, seed, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    density = min(1.0, 400.0 / k)            # keeps |T| within 8 bits
    x, w = ints(gen, tokens, k, density=density), ints(gen, n, k, lo=-2, hi=2)
    a, b = ints(gen, adapters, rank, k), ints(gen, adapters, n, rank)
    scale = 2.0 ** torch.randint(-1, 2, (adapters,), generator=gen, device="cuda").double()
    adapter = ids_for(kind, tokens, adapters, gen)
    t = x @ a.flatten(0, 1).T
    assert t.abs().max() <= 128
    want = plain(x, w, a, b, adapter.long(), scale)
    assert want.abs().max() < 2 ** 22
    cast = [padded(v.to(dtype)) for v in (x, w, a, b)]
    return cast + [adapter, scale.float()], want


def check_exact(tokens, n, k, rank, adapters, kind, dtype=torch.bfloat16, out=torch.float32, seed=1, **plan_kw):
    tensors, want = make_exact(tokens, n, k, rank, adapters, kind, seed, dtype)
    x, w, a, b, adapter, scale = tensors
    y = padded(torch.full((tokens, n), NAN, dtype=out, device="cuda"))
    with dg.LoraPlan(tokens, n, k, rank=rank, adapters=adapters, dtype=CODE[dtype], dtype_y=CODE[out], ldx=x.stride(0), ldw=w.stride(0),
                     ldy=y.stride(0), **plan_kw) as plan:
        for _ in range(2):                   # the second run meets the first one's workspace
            y.fill_(NAN)
            plan.run(x, w, a, b, adapter, y, scale=scale)
            s, rec = plan.sync_status()
            assert s == dg.GEMM_OK, (dg.gemm_status_string(s), rec.role, rec.stage, rec.tile)
            assert torch.equal(y, want.to(out)), (y.double() - want.to(out).double()).abs().max()
        assert torch.isnan(y._base[:, n:]).all()          # the padding behind the rows is not written
        return plan.info


@pytest.mark.parametrize("kind", ["none", "one", "runs", "mixed", "wild"])
@pytest.mark.parametrize("tokens", [1, 3, 8, 9, 96, 128, 129, 256, 257, 700])
def test_tokens_and_adapter_patterns(tokens, kind):
    check_exact(tokens, 264, 328, 16, 7, kind)


@pytest.mark.parametrize("rank", [8, 16, 24, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("tokens", [5, 300])
def test_ranks(tokens, rank):
    check_exact(tokens, 200, 192, rank, 3, "mixed")


@pytest.mark.parametrize("n,k", [(1, 1), (3, 7), (8, 64), (129, 63), (257, 1001), (1543, 65), (40, 4104), (4096, 512), (8200, 128)])
@pytest.mark.parametrize("tokens", [2, 130, 515])
def test_ragged_sizes(tokens, n, k):
    check_exact(tokens, n, k, 16, 4, "mixed")


@pytest.mark.parametrize("dtype,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float16), (torch.float16, torch.float16),
                                       (torch.float16, torch.bfloat16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("tokens", [6, 300])
def test_types(tokens, dtype, out):
    check_exact(tokens, 321, 200, 24, 5, "mixed", dtype=dtype, out=out)


@pytest.mark.parametrize("adapters", [1, 2, 31, 32, 33, 200, 1000, 4096])
@pytest.mark.parametrize("tokens", [64, 400])
def test_many_adapters(tokens, adapters):
    check_exact(tokens, 72, 72, 8, adapters, "mixed")


@pytest.mark.parametrize("kw", [dict(flags=dg.GEMM_FLAG_CTA_GROUP_1), dict(flags=dg.GEMM_FLAG_CTA_GROUP_2),
                                dict(flags=dg.GEMM_FLAG_NO_STREAM_K), dict(flags=dg.GEMM_FLAG_STAGE_K1),
                                dict(flags=dg.GEMM_FLAG_CTA_GROUP_2 | dg.GEMM_FLAG_STAGE_K2), dict(tile_n=64), dict(tile_n=256),
                                dict(tile_n=512), dict(tile_n=512, flags=dg.GEMM_FLAG_CTA_GROUP_2), dict(max_ctas=3), dict(stages=2)])
@pytest.mark.parametrize("tokens,n,k", [(40, 300, 8200), (600, 1100, 1030)])
def test_persistent_kernel_choices(tokens, n, k, kw):
    """Forced tiles, CTA groups, stage depths and splits (40 x 300 x 8200 splits its few tiles along K) give the same Y."""
    info = check_exact(tokens, n, k, 24, 6, "mixed", **kw)
    assert info.product_k_split == 1


@pytest.mark.parametrize("rank,kind", [(16, "runs"), (64, "runs"), (24, "mixed")])
def test_wide_tiles(rank, kind):
    """512-wide tiles, whose halves are handed back apart: the steps join both before the left one goes (65 K blocks: the split
    schedule; 5: the plain one)."""
    info = check_exact(2100, 4104, 4104, rank, 5, kind, out=torch.bfloat16, tile_n=512, flags=dg.GEMM_FLAG_CTA_GROUP_2)
    assert info.product.tile_n == 512
    check_exact(700, 1030, 300, rank, 5, kind, out=torch.bfloat16, tile_n=512, flags=dg.GEMM_FLAG_CTA_GROUP_2)


def test_clusters_split_k_and_steps():
    """Few tiles: clusters of CTAs, more adapter steps than the ring holds, fewer K blocks than CTAs in a cluster."""
    info = check_exact(100, 512, 4096, 64, 90, "mixed")
    assert info.product_k_split > 1
    check_exact(128, 64, 130, 128, 128, "mixed")
    check_exact(20, 64, 64, 16, 20, "mixed")


@pytest.mark.parametrize("tokens,n,k,adapters,kind", [
    (257, 200, 2056, 4, "runs"), (300, 1030, 2100, 3, "one"), (512, 136, 2100, 40, "mixed"), (511, 4100, 2048, 60, "wild"),       # few tiles, long K
    (513, 136, 2100, 4, "runs"), (1000, 520, 136, 200, "mixed"), (1024, 300, 4200, 64, "mixed"), (1025, 300, 200, 64, "mixed"),   # persistent, gathered or streamed
    (777, 2100, 3200, 300, "wild")])
def test_middle_sizes(tokens, n, k, adapters, kind):
    """Around the token counts at which the kernels of both launches change."""
    check_exact(tokens, n, k, 24, adapters, kind, out=torch.bfloat16)


def test_workspace_carries_nothing_over():
    """One plan, adapters that change from run to run: rows that had an adapter's T must be zero for it now."""
    for tokens in (60, 500):
        plan = None
        for seed, kind in ((1, "one"), (2, "mixed"), (3, "none"), (4, "runs"), (5, "wild")):
            (x, w, a, b, adapter, scale), want = make_exact(tokens, 136, 200, 16, 9, kind, seed, torch.bfloat16)
            if plan is None:
                plan = dg.LoraPlan(tokens, 136, 200, rank=16, adapters=9, dtype_y=dg.GEMM_F32, ldx=x.stride(0), ldw=w.stride(0))
            y = torch.empty(tokens, 136, device="cuda")
            plan.run(x, w, a, b, adapter, y, scale=scale)
            assert torch.equal(y, want.float()), (tokens, kind)
        plan.close()


@pytest.mark.parametrize("tokens", [20, 300])
def test_one_token_s_nan_stays_its_own(tokens):
    (x, w, a, b, adapter, scale), want = make_exact(tokens, 96, 128, 16, 4, "mixed", 3, torch.bfloat16)
    adapter[5], adapter[11] = 2, 2
    want = plain(x.double(), w.double(), a.double(), b.double(), adapter.long(), scale.double())
    x[5, 7], x[11, 100] = NAN, float("inf")
    # an adapter that no token uses
    adapter[adapter == 1] = -1
    want = plain(torch.nan_to_num(x.double(), 0, 0), w.double(), a.double(), b.double(), adapter.long(), scale.double())
    a[1], b[1] = NAN, NAN
    y = torch.empty(tokens, 96, device="cuda")
    with dg.LoraPlan(tokens, 96, 128, rank=16, adapters=4, dtype_y=dg.GEMM_F32, ldx=x.stride(0), ldw=w.stride(0)) as plan:
        plan.run(x, w, a, b, adapter, y, scale=scale)
        torch.cuda.synchronize()
    others = torch.ones(tokens, dtype=torch.bool, device="cuda")
    others[[5, 11]] = False
    assert torch.equal(y[others], want.float()[others])
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[11]).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,n,k,rank,kw", [
    (20, 96, 128, 16, {}), (200, 264, 2056, 24, {}), (300, 1030, 2100, 16, {}), (300, 250, 96, 136, {}),
    (700, 520, 200, 16, dict(flags=dg.GEMM_FLAG_CTA_GROUP_1)), (700, 520, 200, 16, dict(flags=dg.GEMM_FLAG_CTA_GROUP_2)),
    (40, 300, 8200, 16, dict(tile_n=64)), (600, 1100, 1030, 16, dict(tile_n=512, flags=dg.GEMM_FLAG_CTA_GROUP_2))])
def test_one_adapter_s_nan_stays_its_own(tokens, n, k, rank, kw, out):
    """Infinities and NaN in an adapter reach the tokens that use it and no others, though they share its tiles: columns of B,
    one whole A, and their neighbours with neither."""
    (x, w, a, b, adapter, scale), want = make_exact(tokens, n, k, rank, 5, "mixed", 3, torch.bfloat16)
    b[2, 3], b[2, n - 1, 1], b[4, ::7], a[1] = NAN, float("inf"), -float("inf"), NAN
    y = padded(torch.empty(tokens, n, dtype=out, device="cuda"))
    with dg.LoraPlan(tokens, n, k, rank=rank, adapters=5, dtype_y=CODE[out], ldx=x.stride(0), ldw=w.stride(0), ldy=y.stride(0),
                     **kw) as plan:
        for _ in range(2):
            y.fill_(7)
            plan.run(x, w, a, b, adapter, y, scale=scale)
            assert plan.sync_status()[0] == dg.GEMM_OK
            same = y == want.to(out)
            hit = torch.zeros(5, n, dtype=torch.bool, device="cuda")       # columns of an adapter's tokens that may differ
            hit[1], hit[2, 3], hit[2, n - 1], hit[4, ::7] = True, True, True, True
            may = (adapter >= 0)[:, None] & hit[adapter.clamp(min=0).long()]
            assert same[~may].all()
            assert torch.isnan(y[adapter == 1]).all() and torch.isnan(y[adapter == 2, 3]).all()
            assert not torch.isfinite(y[adapter == 4][:, ::7]).any()


@pytest.mark.parametrize("tokens,n,k,rank,adapters,kind,dtype,out", [
    (1, 4096, 4096, 16, 8, "one", torch.bfloat16, torch.bfloat16), (77, 1000, 2048, 32, 40, "mixed", torch.bfloat16, torch.bfloat16),
    (200, 777, 3001, 64, 6, "mixed", torch.float16, torch.float16), (1500, 1024, 1024, 16, 3, "runs", torch.bfloat16, torch.float32),
    (90, 512, 4096, 128, 12, "mixed", torch.bfloat16, torch.float32)])
def test_random_inputs(tokens, n, k, rank, adapters, kind, dtype, out):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    x, w = torch.randn(tokens, k, generator=gen, device="cuda"), torch.randn(n, k, generator=gen, device="cuda") * k ** -0.5
    a, b = torch.randn(adapters, rank, k, generator=gen, device="cuda") * k ** -0.5, torch.randn(adapters, n, rank, generator=gen, device="cuda")
    x, w, a, b = (padded(v.to(dtype)) for v in (x, w, a, b))
    scale = torch.rand(adapters, generator=gen, device="cuda") + 0.5
    adapter = ids_for(kind, tokens, adapters, gen)
    y = padded(torch.empty(tokens, n, dtype=out, device="cuda"))
    with dg.LoraPlan(tokens, n, k, rank=rank, adapters=adapters, dtype=CODE[dtype], dtype_y=CODE[out], ldx=x.stride(0), ldw=w.stride(0),
                     ldy=y.stride(0)) as plan:
        plan.run(x, w, a, b, adapter, y, scale=scale)
        first = y.clone()
        plan.run(x, w, a, b, adapter, y, scale=scale)
        assert torch.equal(first, y)                      # fixed summation orders
    xd, wd, ad, bd, sd = x.double(), w.double(), a.double(), b.double(), scale.double()
    want = plain(xd, wd, ad, bd, adapter.long(), sd)
    total = plain(xd.abs(), wd.abs(), ad.abs(), bd.abs(), adapter.long(), sd)
    delta = torch.zeros_like(want)
    for i in range(adapters):
        rows = (adapter == i).nonzero().flatten()
        if len(rows):
            delta[rows] = sd[i] * ((xd[rows] @ ad[i].T).abs() @ bd[i].abs().T)
    u = U[dtype] ** (2 if out == torch.float32 else 1)
    inner = (k / 8 + 16) * 2.0 ** -23 * total + u * delta
    allowed = inner + U[out] * (want.abs() + inner)
    assert ((y.double() - want).abs() <= allowed).all(), ((y.double() - want).abs() / allowed).max()


def test_adapters_in_a_pool_with_their_own_strides():
    (x, w, a, b, adapter, scale), want = make_exact(50, 120, 88, 16, 5, "mixed", 9, torch.bfloat16)
    pool_a = torch.full((12, 20, 104), NAN, dtype=torch.bfloat16, device="cuda")
    pool_b = torch.full((12, 128, 24), NAN, dtype=torch.bfloat16, device="cuda")
    va, vb = pool_a[1:11:2, 2:18, 8:96], pool_b[1:11:2, :120, 8:]
    va.copy_(a)
    vb.copy_(b)
    y = torch.empty(50, 120, device="cuda")
    with dg.LoraPlan(50, 120, 88, rank=16, adapters=5, dtype_y=dg.GEMM_F32, ldx=x.stride(0), ldw=w.stride(0)) as plan:
        plan.run(x, w, va, vb, adapter, y, scale=scale)
    assert torch.equal(y, want.float())


def test_other_streams_graphs_and_no_scale():
    (x, w, a, b, adapter, scale), _ = make_exact(33, 128, 256, 16, 4, "mixed", 2, torch.bfloat16)
    want = plain(x.double(), w.double(), a.double(), b.double(), adapter.long(), torch.ones(4, dtype=torch.double, device="cuda")).float()
    y = torch.zeros(33, 128, device="cuda")
    plan = dg.LoraPlan(33, 128, 256, rank=16, adapters=4, dtype_y=dg.GEMM_F32, ldx=x.stride(0), ldw=w.stride(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.run(x, w, a, b, adapter, y)
    side.synchronize()
    assert torch.equal(y, want)
    y.zero_()
    torch.cuda.synchronize()
    plan.run(x, w, a, b, adapter, y, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(x, w, a, b, adapter, y)
    for shift in range(3):                   # the captured launch follows the contents of its buffers
        adapter.copy_((adapter + 1 + shift) % 4)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = plain(x.double(), w.double(), a.double(), b.double(), adapter.long(), torch.ones(4, dtype=torch.double, device="cuda")).float()
        assert torch.equal(y, want)
    plan.close()


def test_lora_matmul_and_empty_batches():
    (x, w, a, b, adapter, scale), want = make_exact(21, 64, 72, 8, 3, "mixed", 4, torch.bfloat16)
    y = dg.lora_matmul(x, w, a, b, adapter, scale=scale, out_dtype=torch.float32)
    assert torch.equal(y, want.float())
    assert dg.lora_matmul(x, w, a, b, adapter, scale=scale).dtype == torch.bfloat16
    assert torch.equal(dg.lora_matmul(x[:1], w, a, b, adapter[:1], scale=scale, out_dtype=torch.float32), want.float()[:1])
    none = dg.lora_matmul(x[:0], w, a, b, adapter[:0], scale=scale)
    assert tuple(none.shape) == (0, 64)


def test_lora_matmul_with_ever_new_token_counts(monkeypatch):
    """Plans come and go; a graph's plan stays."""
    from dense_gemm_blackwell_gb300 import serving
    monkeypatch.setattr(serving, "_LORA_PLAN_COUNT", 3)
    (x, w, a, b, adapter, scale), want = make_exact(80, 264, 328, 16, 7, "mixed", 2, torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.empty(33, 264, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dg.lora_matmul(x[:33], w, a, b, adapter[:33], scale=scale, out=out)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            dg.lora_matmul(x[:33], w, a, b, adapter[:33], scale=scale, out=out)
    torch.cuda.synchronize()
    for tokens in (1, 80, 17, 9, 64, 80, 2, 50):
        y = dg.lora_matmul(x[:tokens], w, a, b, adapter[:tokens], scale=scale, out_dtype=torch.float32)
        assert torch.equal(y, want.float()[:tokens])
    assert len(serving._lora_plans) <= 4
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.float()[:33])


@pytest.mark.parametrize("tokens", [40, 700])
def test_lora_matmul_from_several_threads(tokens):
    """Threads that share a stream and a shape, each with inputs of its own."""
    cases = [make_exact(tokens, 264, 328, 16, 7, "mixed", 10 + i, torch.bfloat16) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        (x, w, a, b, adapter, scale), want = cases[i]
        for _ in range(50):
            if not torch.equal(dg.lora_matmul(x, w, a, b, adapter, scale=scale, out_dtype=torch.float32), want.float()):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens", [5, 300, 700])
def test_a_sum_past_f16_is_an_infinity(tokens, out):
    """scale T is rounded to f16: what does not fit is an infinity of its sign in any output type, for its own token only."""
    (x, w, a, b, adapter, scale), _ = make_exact(tokens, 40, 72, 16, 2, "one", 6, torch.float16)
    a.zero_()
    a[:, 0, 0] = 1024.0
    b.copy_(b.abs())
    b[:, :, 0] = 1.0
    x[:, 0] = torch.randint(-2, 3, (tokens,), device="cuda").half()
    x[3, 0], x[4, 0] = 1024.0, -1024.0
    scale.fill_(1.0)
    want = plain(x.double(), w.double(), a.double(), b.double(), adapter.long(), scale.double())
    want[3], want[4] = float("inf"), float("-inf")
    y = torch.empty(tokens, 40, dtype=out, device="cuda")
    with dg.LoraPlan(tokens, 40, 72, rank=16, adapters=2, dtype=dg.GEMM_F16, dtype_y=CODE[out], ldx=x.stride(0), ldw=w.stride(0)) as plan:
        plan.run(x, w, a, b, adapter, y, scale=scale)
        assert plan.sync_status()[0] == dg.GEMM_OK
    assert torch.equal(y, want.to(out))


@pytest.mark.parametrize("n,k", [(1543, 1001), (1, 1001), (7, 3)])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_lora_matmul_takes_single_rows_of_any_width(n, k, out):
    (x, w, a, b, adapter, scale), want = make_exact(1, n, k, 16, 2, "one", 5, torch.bfloat16)
    y = dg.lora_matmul(x.contiguous(), w, a, b, adapter, scale=scale, out_dtype=out)
    assert torch.equal(y, want.to(out))


def test_strides_of_single_elements_do_not_matter():
    (x, w, a, b, adapter, scale), want = make_exact(2, 1, 128, 16, 1, "one", 3, torch.bfloat16)
    y = torch.empty(2, 8, device="cuda")[:, :1]
    with dg.LoraPlan(2, 1, 128, rank=16, adapters=1, dtype_y=dg.GEMM_F32, ldx=x.stride(0), ldy=8) as plan:
        plan.run(x, w.as_strided((1, 128), (1, 1)), a.as_strided(a.shape, (1, a.stride(1), 1)), b.as_strided(b.shape, (1, 3, 1)), adapter, y, scale=scale)
    assert torch.equal(y, want.float())


def test_refusals():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda")
    a, b = torch.zeros(2, 16, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 32, 16, dtype=torch.bfloat16, device="cuda")
    ids, y = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    with dg.LoraPlan(4, 32, 64, rank=16, adapters=2) as plan:
        plan.run(x, w, a, b, ids, y)
        for bad in (dict(x=x.half()), dict(w=w.float()), dict(adapter=ids.long()), dict(y=y.float())):
            with pytest.raises(TypeError):
                plan.run(**{**dict(x=x, w=w, a=a, b=b, adapter=ids, y=y), **bad})
        for bad in (dict(x=x[:3]), dict(w=w.t().contiguous()), dict(a=a[:1]), dict(b=b[:, :16]), dict(adapter=ids[:2]), dict(adapter=ids.cpu()),
                    dict(x=x.t().contiguous().t()), dict(scale=torch.ones(3, device="cuda"))):
            with pytest.raises(ValueError):
                plan.run(**{**dict(x=x, w=w, a=a, b=b, adapter=ids, y=y), **bad})
        wide = torch.zeros(2, 16, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
        with pytest.raises(dg.GemmError) as e:            # rows of A 136 bytes apart
            plan.run(x, w, wide, b, ids, y)
        assert e.value.status == dg.GEMM_ERR_ALIGNMENT
    with pytest.raises(dg.GemmError) as e:
        dg.LoraPlan(4, 32, 64, rank=12, adapters=2)
    assert e.value.status == dg.GEMM_ERR_UNSUPPORTED
