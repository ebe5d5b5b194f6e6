"""GPU: attention of one new token over a paged key-value cache, against a plain 64-bit form.

Tolerances.  With p the softmax and S = sum p |v| (the values' scale included):
  |out - out64| <= (u_p + 2 d + 2^-17) S + f + u (|out64| + the above)
u = 2^-8 (bf16) or 2^-11 (f16): the output's rounding; u_p = u of the type P is rounded to for its product with V (f16 with an
E4M3 cache); d bounds the error of a score: fp32 sums of head_dim exact products, (head_dim + 8) 2^-24 of scale sum |q||k|,
which moves p by a factor of 1 +- 2 d; f = 2^-40 sum |v| where P is f16, whose smallest unit is 2^-24 of 2^15 times the
probabilities relative to the row's largest (an E4M3 value of exactly zero can leave S to probabilities below it); 2^-17 covers the exponentials (2^-22 each, a few rescalings) and fp32 sums.  bf16
queries against an E4M3 cache are scaled to f16 by a power of two: elements 2^-14 below a row's largest lose bits, at most
2^-24 of the largest each, so d grows by head_dim 2^-24 scale max|q| max|k|.
  |lse - lse64| <= d + 2^-20 (1 + |lse64|).
"""
import math

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

CODE = {torch.bfloat16: dg.GEMM_BF16, torch.float16: dg.GEMM_F16, torch.float8_e4m3fn: dg.GEMM_E4M3}
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E4M3 = torch.float8_e4m3fn
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def make(lengths, heads, kv, dim, page, dtype, cache, seed=0, layout="pages", extra=3, tail=NAN):
    """Inputs whose cache holds `tail` wherever no sequence has a position."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    used = [-(-n // page) for n in lengths]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=gen, device="cuda").tolist()
    width = max(max(used), 1) + 2
    table = torch.full((len(lengths), width), -1, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = torch.tensor(order[at: at + u], dtype=torch.int32)
        at += u
    shape = (pages, page, kv, dim) if layout == "pages" else (pages, kv, page, dim)
    caches = []
    for _ in range(2):
        c = r(*shape) * (1 if cache != E4M3 else 30)
        c = c if layout == "pages" else c.permute(0, 2, 1, 3)
        keep = torch.zeros(pages, page, dtype=torch.bool)
        for i, n in enumerate(lengths):
            for j in range(used[i]):
                keep[table[i, j], : min(page, n - j * page)] = True
        c = torch.where(keep.cuda()[:, :, None, None], c, torch.tensor(tail, device="cuda"))
        caches.append(c.to(cache))
        if layout != "pages":
            assert not caches[-1].is_contiguous()
    q = (r(len(lengths), heads * dim + 16) * 1.5).to(dtype)[:, : heads * dim].unflatten(1, (heads, dim))
    return q, caches[0], caches[1], table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda")


def plain(q, kc, vc, table, lengths, window, scale, ks, vs):
    """(out, S, lse, d, f) in 64 bits; S, d and f as in the head of this file."""
    b, heads, dim = q.shape
    kv, page = kc.shape[2], kc.shape[1]
    group = heads // kv
    out = torch.zeros(b, heads, dim, dtype=torch.double, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((b, heads), -math.inf, dtype=torch.double, device="cuda")
    d, f = torch.zeros(b, heads, dtype=torch.double, device="cuda"), torch.zeros_like(out)
    for i, n in enumerate(lengths.tolist()):
        n = max(0, min(n, table.shape[1] * page))
        pos = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        pages = table[i, pos // page].long()
        valid = (pages >= 0) & (pages < kc.shape[0])
        pos, pages = pos[valid], pages[valid]
        if len(pos) == 0:
            continue
        k, v = kc[pages, pos % page].double() * ks, vc[pages, pos % page].double() * vs          # [n, kv, dim]
        for h in range(heads):
            s = (k[:, h // group] @ q[i, h].double()) * scale
            absum = (k[:, h // group].abs() @ q[i, h].double().abs()) * abs(scale)
            finite = torch.isfinite(absum)
            d[i, h] = (dim + 8) * 2.0 ** -24 * absum[finite].max() if finite.any() else 0
            if q.dtype == torch.bfloat16 and kc.dtype == E4M3:
                d[i, h] += dim * 2.0 ** -24 * abs(scale) * q[i, h].double().abs().max() * k[:, h // group].abs().max()
            lse[i, h] = torch.logsumexp(s, 0)
            if lse[i, h] == -math.inf:
                continue
            p = torch.softmax(s, 0)
            out[i, h], mag[i, h] = p @ v[:, h // group], p @ v[:, h // group].abs()
            if kc.dtype != torch.bfloat16:
                f[i, h] = 2.0 ** -40 * v[:, h // group].abs().sum(0)
    return out, mag, lse, d, f


def check(q, kc, vc, table, lengths, window=0, scale=None, ks=1.0, vs=1.0, max_ctas=0, plan=None):
    heads, dim = q.shape[1:]
    out = torch.full((q.shape[0], heads * dim + 8), NAN, dtype=q.dtype, device="cuda")[:, : heads * dim].unflatten(1, (heads, dim))
    lse = torch.full((q.shape[0], heads), NAN, device="cuda")
    own = plan is None
    if own:
        plan = dg.PagedAttentionPlan(q.shape[0], heads=heads, kv_heads=kc.shape[2], head_dim=dim, page_size=kc.shape[1], dtype=CODE[q.dtype],
                                     dtype_cache=CODE[kc.dtype], window=window, max_ctas=max_ctas)
    plan.run(q, kc, vc, table, lengths, out, lse=lse, scale=scale, k_scale=ks, v_scale=vs)
    again = torch.empty_like(q, memory_format=torch.contiguous_format)
    plan.run(q, kc, vc, table, lengths, again, scale=scale, k_scale=ks, v_scale=vs)      # counters are back at zero, order is fixed
    assert torch.equal(again.view(torch.int16), out.contiguous().view(torch.int16))
    if own:
        plan.close()
    scale = dim ** -0.5 if scale is None else scale
    want, mag, wl, d, f = plain(q, kc, vc, table, lengths, window, scale, ks, vs)
    u = U[q.dtype]
    up = U[torch.float16] if kc.dtype == E4M3 else u
    inner = (up + 2 * d[..., None] + 2.0 ** -17) * mag + f
    allowed = inner + u * (want.abs() + inner)
    err = (out.double() - want).abs()
    assert (err <= allowed).all(), (err / allowed.clamp(min=1e-300)).max()
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert ((lse.double() - wl).abs()[~empty] <= (d + 2.0 ** -20 * (1 + wl.abs()))[~empty]).all()
    return out


EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("page", [1, 7, 8, 16, 24, 64, 100])
@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, E4M3), (torch.float16, E4M3)])
def test_lengths_and_pages(page, dtype, cache):
    check(*make(EDGES, 8, 2, 64, page, dtype, cache, seed=page), ks=0.02 if cache == E4M3 else 1.0, vs=0.03 if cache == E4M3 else 1.0)


@pytest.mark.parametrize("dim", [8, 24, 40, 64, 72, 80, 96, 104, 112, 128, 136, 192, 256])
@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float16, E4M3])
def test_head_sizes(dim, cache):
    if cache == E4M3 and dim % 16:
        dim += 8
    dtype = torch.float16 if cache == torch.float16 else torch.bfloat16
    check(*make([0, 5, 130, 700], 6, 3, dim, 16, dtype, cache, seed=dim), ks=0.02 if cache == E4M3 else 1.0)


@pytest.mark.parametrize("group", [1, 2, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("kv", [1, 3])
def test_shared_heads(kv, group):
    check(*make([1, 77, 300], kv * group, kv, 128, 16, torch.bfloat16, torch.bfloat16, seed=group))


@pytest.mark.parametrize("window", [1, 16, 63, 64, 100, 1000])
@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
def test_windows(window, cache):
    q, kc, vc, table, lengths = make([0, 1, 50, 64, 129, 999, 1000, 1001], 8, 2, 80, 24, torch.bfloat16, cache, seed=window)
    for i, n in enumerate(lengths.tolist()):             # nothing before the window is read into the result
        for j in range(max(0, n - window) // 24):
            kc[table[i, j].long()], vc[table[i, j].long()] = torch.tensor(NAN).to(cache).cuda(), torch.tensor(NAN).to(cache).cuda()
    check(q, kc, vc, table, lengths, window=window)


@pytest.mark.parametrize("max_ctas", [0, 1, 2, 7, 40])
@pytest.mark.parametrize("dim,group,cache", [(128, 4, torch.bfloat16), (64, 12, torch.float16), (80, 3, E4M3), (256, 2, torch.bfloat16)])
def test_long_sequences_are_split_and_joined(dim, group, cache, max_ctas):
    """One long sequence among short and empty ones; few CTAs walk many segments, many CTAs share one."""
    dtype = torch.float16 if cache == torch.float16 else torch.bfloat16
    check(*make([3, 6001, 0, 0, 130, 1, 2500], 2 * group, 2, dim, 16, dtype, cache, seed=dim), max_ctas=max_ctas)


def test_many_sequences():
    gen = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 90, (700,), generator=gen).tolist()
    check(*make(lengths, 4, 2, 64, 8, torch.bfloat16, torch.bfloat16))
    check(*make([0] * 300, 4, 2, 64, 8, torch.bfloat16, torch.bfloat16))
    check(*make([0] * 299 + [40], 4, 2, 64, 8, torch.bfloat16, torch.bfloat16))


def test_head_major_cache_and_shared_buffer():
    check(*make([1, 100, 513], 8, 4, 96, 16, torch.bfloat16, torch.bfloat16, layout="heads first"))
    check(*make([1, 100, 513], 8, 4, 96, 16, torch.float16, E4M3, layout="heads first"), ks=0.05, vs=0.02)
    q, kc, vc, table, lengths = make([9, 300], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    both = torch.stack((kc, vc), 2)                      # keys and values of a page place side by side
    check(q, both[:, :, 0], both[:, :, 1], table, lengths)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_scales(scale):
    check(*make([1, 40, 333], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16), scale=scale)


def test_lengths_out_of_range_and_pages_that_do_not_exist():
    q, kc, vc, table, lengths = make([40, 90, 200, 64], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16, tail=0.5)
    lengths[0] = -3                                      # as 0
    lengths[3] = 10 ** 9                                 # clamped to the table; its unused columns hold -1: masked
    table[1, 2], table[1, 3], table[2, 0] = -1, 10 ** 6, kc.shape[0]
    out = check(q, kc, vc, table, lengths)
    assert torch.equal(out[0], torch.zeros_like(out[0]))
    table[2] = -1                                        # a sequence none of whose pages exist
    out = check(q, kc, vc, table, lengths)
    assert torch.equal(out[2], torch.zeros_like(out[2]))


def test_infinite_scores():
    """Keys at minus infinity: their positions get nothing; where all are, the output is zero and the sum's logarithm -inf."""
    q, kc, vc, table, lengths = make([70, 33], 2, 1, 64, 16, torch.bfloat16, torch.bfloat16)
    q[..., 0] = 1.0
    kc[..., 0] = torch.where(torch.rand(kc.shape[:3], device="cuda") < 0.5, -math.inf, 0.0).to(torch.bfloat16)
    for j in range(3):
        kc[table[1, j].long(), :, :, 0] = -math.inf
    out = check(q, kc, vc, table, lengths)
    assert torch.equal(out[1], torch.zeros_like(out[1]))


@pytest.mark.parametrize("page", [1, 2, 7, 8, 16, 24])
@pytest.mark.parametrize("window", [0, 21])
@pytest.mark.parametrize("dim,dtype,cache", [(64, torch.bfloat16, torch.bfloat16), (128, torch.float16, torch.float16), (64, torch.bfloat16, E4M3),
                                             (128, torch.float16, E4M3)])
def test_a_page_named_by_neighbouring_columns(dim, dtype, cache, window, page):
    """Columns that name one page: each position reads its own place of it, the cache's last page among them."""
    gen = torch.Generator(device="cuda").manual_seed(page)
    pages, width = 5, -(-150 // page)
    kc, vc = ((torch.randn(pages, page, 2, dim, generator=gen, device="cuda") * (30 if cache == E4M3 else 1)).to(cache) for _ in range(2))
    q = torch.randn(4, 8, dim, generator=gen, device="cuda").to(dtype)
    col = torch.arange(width, device="cuda")
    last = torch.full_like(col, pages - 1)
    table = torch.stack((last, col // 2 % pages, torch.where(col < 3, 1, last), torch.where(col % 2 == 0, last, 0))).to(torch.int32)
    lengths = torch.tensor([150, 149, 96, 32], dtype=torch.int32, device="cuda")
    check(q, kc, vc, table, lengths, window=window, ks=0.02 if cache == E4M3 else 1.0, vs=0.03 if cache == E4M3 else 1.0)


def test_large_scores():
    """Softmax far from its mean: one key dominates by hundreds."""
    q, kc, vc, table, lengths = make([500, 64], 4, 2, 128, 16, torch.bfloat16, torch.bfloat16)
    check(q, kc, vc, table, lengths, scale=3.0)


def test_batch_smaller_than_the_plan_and_empty_batch():
    q, kc, vc, table, lengths = make([5, 100, 64, 200], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    plan = dg.PagedAttentionPlan(9, heads=4, kv_heads=2, head_dim=64, page_size=16)
    for n in (4, 1, 3, 2):
        check(q[:n], kc, vc, table[:n], lengths[:n], plan=plan)
    plan.run(q[:0], kc, vc, table[:0], lengths[:0], torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"))
    plan.close()


def test_cache_beyond_32_bits():
    """Pages whose element offsets pass 2^31 (a 4.7 GB cache each)."""
    pages, page, kv, dim = 72000, 16, 8, 256
    kc, vc = (torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[71999, 65537, 70001, 0, 65536], [3, 71998, 1, 2, 70000]], dtype=torch.int32, device="cuda")
    for c in (kc, vc):
        c[table.flatten().long()] = torch.randn(10, page, kv, dim, device="cuda").to(torch.bfloat16)
    q = torch.randn(2, 16, dim, device="cuda").to(torch.bfloat16)
    check(q, kc, vc, table, torch.tensor([77, 80], dtype=torch.int32, device="cuda"))


def test_strides_of_single_elements_do_not_matter():
    q, kc, vc, table, lengths = make([77], 4, 1, 64, 16, torch.bfloat16, torch.bfloat16)
    want = check(q, kc, vc, table, lengths)
    odd = lambda t, *strides: t.as_strided(t.shape, strides)  # noqa: E731
    q, kc, vc = odd(q.contiguous(), 1, 64, 1), odd(kc, 1024, 64, 3, 1), odd(vc, 1024, 64, 1, 1)
    assert torch.equal(check(q, kc, vc, odd(table, 1, 1), lengths), want)


def test_streams_and_graph():
    q, kc, vc, table, lengths = make([500, 64, 0, 1000], 8, 2, 128, 16, torch.bfloat16, torch.bfloat16)
    plan = dg.PagedAttentionPlan(4, heads=8, kv_heads=2, head_dim=128, page_size=16)
    want = check(q, kc, vc, table, lengths, plan=plan).contiguous()
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.run(q, kc, vc, table, lengths, out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(q, kc, vc, table, lengths, out)
    for n in ([500, 64, 0, 1000], [1, 2, 3, 4], [0, 0, 0, 0], [33, 600, 128, 999]):      # the captured launch follows the lengths
        lengths.copy_(torch.tensor([min(a, b) for a, b in zip(n, (500, 64, 0, 1000))], dtype=torch.int32))
        out.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, check(q, kc, vc, table, lengths, plan=plan))
    plan.close()


def test_refusals():
    q, kc, vc, table, lengths = make([5, 6], 4, 2, 64, 16, torch.bfloat16, torch.bfloat16)
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    plan = dg.PagedAttentionPlan(2, heads=4, kv_heads=2, head_dim=64, page_size=16)
    good = dict(q=q, k_cache=kc, v_cache=vc, block_table=table, lengths=lengths, out=out)
    plan.run(**good)
    for bad in (dict(q=q.half()), dict(k_cache=kc.half()), dict(block_table=table.long()), dict(lengths=lengths.long()), dict(out=out.float()),
                dict(lse=torch.zeros(2, 4, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            plan.run(**{**good, **bad})
    for bad in (dict(q=torch.cat((q, q))), dict(q=q[:, :2]), dict(k_cache=kc[:, :8]), dict(v_cache=vc[:-1]), dict(lengths=lengths[:1]),
                dict(lengths=lengths.cpu()), dict(out=out[:1]), dict(k_cache=kc.transpose(2, 3)), dict(lse=torch.zeros(4, 2, device="cuda"))):
        with pytest.raises(ValueError):
            plan.run(**{**good, **bad})
    for bad in (dict(scale=math.inf), dict(k_scale=NAN)):
        with pytest.raises(dg.GemmError) as e:
            plan.run(**{**good, **bad})
        assert e.value.status == dg.GEMM_ERR_INVALID_ARG
    odd = torch.zeros(kc.numel() + 8, dtype=torch.bfloat16, device="cuda")[1: 1 + kc.numel()].view_as(kc)
    with pytest.raises(dg.GemmError) as e:
        plan.run(**{**good, "k_cache": odd})
    assert e.value.status == dg.GEMM_ERR_ALIGNMENT
    plan.close()
