"""GPU: head norms with rotary positions, their cache append and their backward pass, against a plain 64-bit form.

Tolerances.  u = 2^-8 (bf16), 2^-11 (f16) is the one rounding of an output.  Everything before it is fp32: the row's sum of
squares (at most 256 terms), rsqrt (2 units), the prepared factors w c, w s and two products, about 20 roundings of
2^-24 relative to the magnitudes added, so 2^-18 (64 units) of m = |n_a w_a c| + |n_b w_b s|:
  forward   y is the rounding of some value in [y64 - 2^-18 m, y64 + 2^-18 m]: it lies between the ends' roundings
            (which holds for subnormal f16 outputs as well, whose rounding is not relative)
  backward  |dx - dx64| <= 2^-17 M + u (|dx64| + 2^-17 M),  M = r (|g w| + |n| mean|g w n|),
            twice the forward's allowance for twice the steps (and g's own: 2^-18 of its |dy_a c| + |dy_b s| enters M)
  dweight   fp32 sums over the rows in a tree of at most rows / lane groups + 200 sequential additions: 2^-14 sum |g n|.
E4M3 cache entries: the fp32 value before rounding is off by at most 2^-18 m / scale, so the code is that of some value in
that interval: between the codes of its ends.
"""
import math
import threading

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -18
EPS = 1e-5
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def split_index(rot, interleaved, device="cuda"):
    first = torch.arange(0, rot, 2, device=device) if interleaved else torch.arange(rot // 2, device=device)
    return first, first + (1 if interleaved else rot // 2)


def plain(x, weight, positions, table, interleaved, norm=True):
    """(y, m): the forward result in 64 bits and the magnitudes that add up to it."""
    x = x.double()
    n = x * (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt() if norm else x
    if weight is not None:
        n = n * weight.double()
    t = table.double()[positions.long()]
    rot = 2 * table.shape[2]
    ia, ib = split_index(rot, interleaved)
    c, s = t[:, None, 0], t[:, None, 1]
    y, m = n.clone(), n.abs()
    y[..., ia], y[..., ib] = n[..., ia] * c - n[..., ib] * s, n[..., ia] * s + n[..., ib] * c
    m[..., ia] = (n[..., ia] * c).abs() + (n[..., ib] * s).abs()
    m[..., ib] = (n[..., ia] * s).abs() + (n[..., ib] * c).abs()
    return y, m


def close(got, y, m, u):
    assert got.shape == y.shape and U[got.dtype] == u
    lo, hi = (y - E * m).to(got.dtype).double(), (y + E * m).to(got.dtype).double()
    bad = (got.double() < lo) | (got.double() > hi)
    assert not bad.any(), (got[bad], y[bad])


def make(tokens, heads, kv, dim, rot, dtype, seed=0, weights=True, positions=500):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    qkv = (r(tokens, (heads + 2 * kv) * dim + 8) * 3).to(dtype)          # rows side by side, padded
    q = qkv[:, : heads * dim].unflatten(1, (heads, dim))
    k = qkv[:, heads * dim: (heads + kv) * dim].unflatten(1, (kv, dim))
    v = qkv[:, (heads + kv) * dim: (heads + 2 * kv) * dim].unflatten(1, (kv, dim))
    pos = torch.randint(0, positions, (tokens,), generator=gen, device="cuda").to(torch.int32)
    table = dg.rope_table(positions, rot)
    wq, wk = ((1 + 0.3 * r(dim)).to(dtype), (1 + 0.3 * r(dim)).to(dtype)) if weights else (None, None)
    return q, k, v, pos, table, wq, wk


SHAPES = [  # dim, rot: all lane layouts, rotated parts on and off their boundaries
    (8, 8), (16, 4), (40, 20), (64, 64), (64, 24), (64, 2), (72, 48), (80, 32), (80, 80), (96, 96), (112, 56), (128, 128), (128, 64), (128, 20),
    (136, 96), (192, 128), (256, 256), (256, 64), (256, 10)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_forward_layouts(dim, rot, interleaved, dtype):
    q, k, v, pos, table, wq, wk = make(37, 5, 2, dim, rot, dtype, seed=dim + rot)
    qo, ko = dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, interleaved=interleaved)
    close(qo, *plain(q, wq, pos, table, interleaved), U[dtype])
    close(ko, *plain(k, wk, pos, table, interleaved), U[dtype])


@pytest.mark.parametrize("norm,weights", [(True, False), (False, False), (True, True)])
@pytest.mark.parametrize("tokens,heads,kv", [(1, 1, 1), (1, 32, 8), (3, 7, 7), (1000, 12, 1), (4099, 8, 8)])
def test_forward_sizes(tokens, heads, kv, norm, weights):
    q, k, v, pos, table, wq, wk = make(tokens, heads, kv, 64, 64, torch.bfloat16, seed=tokens, weights=weights)
    qo, ko = dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, norm=norm)
    close(qo, *plain(q, wq, pos, table, False, norm), U[torch.bfloat16])
    close(ko, *plain(k, wk, pos, table, False, norm), U[torch.bfloat16])


def test_queries_alone_in_place_and_without_tokens():
    q, k, v, pos, table, wq, wk = make(50, 4, 2, 128, 64, torch.bfloat16)
    y, m = plain(q, wq, pos, table, False)
    qo, ko = dg.qk_norm_rope(q, None, pos, table, q_weight=wq, eps=EPS)
    assert ko is None
    close(qo, y, m, U[torch.bfloat16])
    yk, mk = plain(k, wk, pos, table, False)
    before_v = v.clone()
    dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, q_out=q, k_out=k)        # over the projection's output
    assert torch.equal(q, qo)
    close(k, yk, mk, U[torch.bfloat16])
    assert torch.equal(v, before_v)
    empty, _ = dg.qk_norm_rope(q[:0], k[:0], pos[:0], table, eps=EPS)
    assert tuple(empty.shape) == (0, 4, 128)


def test_positions_are_clamped_to_the_table():
    q, k, v, pos, table, wq, wk = make(4, 2, 1, 64, 64, torch.bfloat16, positions=10)
    wild = torch.tensor([-5, 10, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    a, _ = dg.qk_norm_rope(q, k, wild, table, eps=EPS)
    b, _ = dg.qk_norm_rope(q, k, wild.clamp(0, 9), table, eps=EPS)
    assert torch.equal(a, b)


def test_zero_rows_and_infinities():
    """A zero row stays zero; without a norm an infinity past the rotated part passes through and touches nothing else."""
    q, k, v, pos, table, wq, wk = make(6, 2, 1, 64, 32, torch.bfloat16, weights=False)
    q[2] = 0
    qo, _ = dg.qk_norm_rope(q, k, pos, table, eps=EPS)
    assert torch.equal(qo[2], torch.zeros_like(qo[2]))
    for interleaved in (False, True):
        for dim, rot in ((64, 32), (64, 20)):
            x = torch.randn(3, 1, dim, device="cuda").to(torch.bfloat16)
            x[1, 0, rot] = float("inf")
            table2 = dg.rope_table(500, rot)
            y, m = plain(torch.where(x.isinf(), 0, x), None, pos[:3], table2, interleaved, norm=False)
            got, _ = dg.qk_norm_rope(x, None, pos[:3], table2, interleaved=interleaved, norm=False)
            assert got[1, 0, rot] == float("inf")
            got[1, 0, rot] = 0
            close(got, y, m, U[torch.bfloat16])


def between_codes(got, lo, hi):
    """Whether every E4M3 value lies between the codes of its interval's ends."""
    f = lambda t: t.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
    return ((got.double() >= f(lo)) & (got.double() <= f(hi))).all()


@pytest.mark.parametrize("layout", ["pages", "heads first"])
@pytest.mark.parametrize("cache_kind", ["same", "e4m3"])
@pytest.mark.parametrize("tokens,page,dim,rot,dtype", [(1, 16, 128, 128, torch.bfloat16), (45, 1, 80, 32, torch.float16),
                                                       (333, 24, 64, 24, torch.bfloat16), (70, 7, 256, 256, torch.float16)])
def test_cache_append(tokens, page, dim, rot, dtype, cache_kind, layout):
    kv = 3
    q, k, v, pos, table, wq, wk = make(tokens, 4, kv, dim, rot, dtype, seed=page)
    pages = tokens // page + 4
    kind = dtype if cache_kind == "same" else torch.float8_e4m3fn
    if layout == "pages":
        caches = [torch.full((pages, page, kv, dim), 7.0, device="cuda").to(kind) for _ in range(2)]
    else:                       # head-major pages, keys and values in one buffer
        both = torch.full((pages, 2, kv, page, dim), 7.0, device="cuda").to(kind)
        caches = [both[:, i].permute(0, 2, 1, 3) for i in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:tokens].to(torch.int32)
    if tokens > 10:
        slots[3], slots[7], slots[9] = -1, pages * page, 2 ** 31 - 1      # nowhere
    scales = dict(k_scale=0.03, v_scale=0.05) if cache_kind == "e4m3" else {}
    qo, ko = dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, v=v, k_cache=caches[0], v_cache=caches[1], slots=slots, **scales)
    assert ko is None
    close(qo, *plain(q, wq, pos, table, False), U[dtype])
    y, m = plain(k, wk, pos, table, False)
    valid = (slots >= 0) & (slots < pages * page)
    where = slots[valid].long()
    flat = [c.reshape(pages * page, kv, dim) if layout == "pages" else c.contiguous().reshape(pages * page, kv, dim) for c in caches]
    if cache_kind == "same":
        close(flat[0][where], y[valid], m[valid], U[dtype])
        assert torch.equal(flat[1][where], v[valid])
    else:
        s = scales["k_scale"]
        slack = E * m[valid] / s + 2.0 ** -23 * (y[valid] / s).abs()
        assert between_codes(flat[0][where], y[valid] / s - slack, y[valid] / s + slack)
        want = (v[valid].float() / torch.tensor(scales["v_scale"], dtype=torch.float32, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(flat[1][where].view(torch.uint8), want.view(torch.uint8))
    untouched = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    untouched[where] = False
    for c in flat:
        assert (c[untouched].double() == torch.tensor(7.0).to(kind).double()).all()


def test_keys_to_buffer_and_cache_at_once():
    q, k, v, pos, table, wq, wk = make(20, 2, 2, 64, 64, torch.bfloat16)
    kc, vc = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(20, dtype=torch.int32, device="cuda") + 9
    _, ko = dg.qk_norm_rope(q, k, pos, table, k_weight=wk, eps=EPS, k_out=torch.empty(20, 2, 64, dtype=torch.bfloat16, device="cuda"), v=v,
                            k_cache=kc, v_cache=vc, slots=slots)
    close(ko, *plain(k, wk, pos, table, False), U[torch.bfloat16])
    assert torch.equal(kc.flatten(0, 1)[9:29], ko)
    assert torch.equal(vc.flatten(0, 1)[9:29], v)


def test_cache_beyond_32_bits():
    """Slots whose element offsets pass 2^31 (a 4.7 GB cache each)."""
    pages, page, kv, dim = 72000, 16, 8, 256
    kc, vc = (torch.empty(pages, page, kv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v, pos, table, wq, wk = make(5, 8, kv, dim, 256, torch.bfloat16)
    slots = torch.tensor([0, 65536 * 16 + 3, pages * page - 1, pages * page - 17, 70000 * 16], dtype=torch.int32, device="cuda")
    dg.qk_norm_rope(q, k, pos, table, k_weight=wk, eps=EPS, v=v, k_cache=kc, v_cache=vc, slots=slots)
    y, m = plain(k, wk, pos, table, False)
    close(kc.flatten(0, 1)[slots.long()], y, m, U[torch.bfloat16])
    assert torch.equal(vc.flatten(0, 1)[slots.long()], v)


# ---------------------------------------------------------------- backward

def plain_backward(x, dy, weight, positions, table, interleaved, norm=True):
    """(dx, M, dweight, sum |g n|) by the formulas, in 64 bits."""
    x, dy = x.double(), dy.double()
    t = table.double()[positions.long()]
    ia, ib = split_index(2 * table.shape[2], interleaved)
    c, s = t[:, None, 0], t[:, None, 1]
    g, gm = dy.clone(), dy.abs()
    g[..., ia], g[..., ib] = dy[..., ia] * c + dy[..., ib] * s, dy[..., ib] * c - dy[..., ia] * s
    gm[..., ia], gm[..., ib] = (dy[..., ia] * c).abs() + (dy[..., ib] * s).abs(), (dy[..., ib] * c).abs() + (dy[..., ia] * s).abs()
    if not norm:
        return g, gm, None, None
    w = torch.ones(x.shape[-1], dtype=torch.double, device="cuda") if weight is None else weight.double()
    r = (x.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    big = r * (gm * w.abs() + n.abs() * (gm * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, big, (g * n).sum((0, 1)), (gm * n.abs()).sum((0, 1))


def close_gradients(got, gw, want, u, weight):
    dx, big, dw, dws = want
    allowed = 2 * E * big + u * (dx.abs() + 2 * E * big)
    assert ((got.double() - dx).abs() <= allowed).all(), ((got.double() - dx).abs() / allowed).max()
    if weight is None:
        assert gw is None
    else:
        assert gw.dtype == torch.float32
        assert ((gw.double() - dw).abs() <= 2.0 ** -14 * dws).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", SHAPES)
def test_backward_layouts(dim, rot, interleaved, dtype):
    q, k, v, pos, table, wq, wk = make(29, 5, 2, dim, rot, dtype, seed=dim * rot)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dq, dk = (torch.randn(t.shape, generator=gen, device="cuda").to(dtype) for t in (q, k))
    gq, gk, gwq, gwk = dg.qk_norm_rope_backward(dq, dk, q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, interleaved=interleaved)
    close_gradients(gq, gwq, plain_backward(q, dq, wq, pos, table, interleaved), U[dtype], wq)
    close_gradients(gk, gwk, plain_backward(k, dk, wk, pos, table, interleaved), U[dtype], wk)


@pytest.mark.parametrize("norm,weights", [(True, False), (False, False), (True, True)])
@pytest.mark.parametrize("tokens,heads,kv", [(1, 1, 1), (3, 7, 7), (1000, 12, 1), (5000, 8, 8), (2, 1, 9)])
def test_backward_sizes(tokens, heads, kv, norm, weights):
    q, k, v, pos, table, wq, wk = make(tokens, heads, kv, 128, 128, torch.bfloat16, seed=tokens, weights=weights)
    dq, dk = torch.randn(q.shape, device="cuda").to(torch.bfloat16), torch.randn(k.shape, device="cuda").to(torch.bfloat16)
    run = lambda: dg.qk_norm_rope_backward(dq, dk, q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, norm=norm)  # noqa: E731
    gq, gk, gwq, gwk = run()
    close_gradients(gq, gwq, plain_backward(q, dq, wq, pos, table, False, norm), U[torch.bfloat16], wq)
    close_gradients(gk, gwk, plain_backward(k, dk, wk, pos, table, False, norm), U[torch.bfloat16], wk)
    for a, b in zip((gq, gk, gwq, gwk), run()):
        assert (a is None and b is None) or torch.equal(a, b)            # fixed summation order


def test_backward_one_weight_queries_alone_and_no_tokens():
    q, k, v, pos, table, wq, wk = make(40, 3, 2, 64, 64, torch.bfloat16)
    dq, dk = torch.randn(q.shape, device="cuda").to(torch.bfloat16), torch.randn(k.shape, device="cuda").to(torch.bfloat16)
    gq, gk, gwq, gwk = dg.qk_norm_rope_backward(dq, dk, q, k, pos, table, k_weight=wk, eps=EPS)
    close_gradients(gq, gwq, plain_backward(q, dq, None, pos, table, False), U[torch.bfloat16], None)
    close_gradients(gk, gwk, plain_backward(k, dk, wk, pos, table, False), U[torch.bfloat16], wk)
    gq, gk, gwq, gwk = dg.qk_norm_rope_backward(dq, None, q, None, pos, table, q_weight=wq, eps=EPS)
    assert gk is None and gwk is None
    close_gradients(gq, gwq, plain_backward(q, dq, wq, pos, table, False), U[torch.bfloat16], wq)
    same = dq.clone()
    dg.qk_norm_rope_backward(same, None, q, None, pos, table, q_weight=wq, eps=EPS, dq_out=same)     # over the incoming gradient
    assert torch.equal(same, gq)
    _, _, gwq, _ = dg.qk_norm_rope_backward(dq[:0], None, q[:0], None, pos[:0], table, q_weight=wq, eps=EPS)
    assert torch.equal(gwq, torch.zeros_like(gwq))


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_against_differences(interleaved):
    """Central differences of the 64-bit forward along random directions d: (L(x + h d) - L(x - h d)) / 2h with h = 1e-5 is the
    derivative to about h^2 times the third derivative plus 2^-52 / h of L, below 1e-6 of sum |dx d| here, against the
    kernel's gradients, whose elements carry one rounding u each (their sum at most u sum |dx d|)."""
    dim, rot = 64, 48
    q, k, v, pos, table, wq, wk = make(6, 2, 1, dim, rot, torch.bfloat16, seed=8)
    dq = torch.randn(q.shape, device="cuda").to(torch.bfloat16)
    gq, _, gw, _ = dg.qk_norm_rope_backward(dq, None, q, None, pos, table, q_weight=wq, eps=EPS, interleaved=interleaved)
    loss = lambda x, w: (plain(x, w, pos, table, interleaved)[0] * dq.double()).sum()  # noqa: E731
    gen = torch.Generator(device="cuda").manual_seed(2)
    h = 1e-5
    for _ in range(20):
        d = torch.randn(q.shape, generator=gen, device="cuda", dtype=torch.double)
        slope = (loss(q.double() + h * d, wq) - loss(q.double() - h * d, wq)) / (2 * h)
        size = (gq.double() * d).abs().sum()
        assert (slope - (gq.double() * d).sum()).abs() <= (2 * U[torch.bfloat16] + 1e-4) * size
        e = torch.randn(dim, generator=gen, device="cuda", dtype=torch.double)
        slope = (loss(q, wq.double() + h * e) - loss(q, wq.double() - h * e)) / (2 * h)
        assert (slope - (gw.double() * e).sum()).abs() <= 1e-4 * (gw.double() * e).abs().sum()


def test_streams_and_graph():
    q, k, v, pos, table, wq, wk = make(64, 4, 2, 128, 128, torch.bfloat16)
    qo, ko = torch.zeros_like(q).contiguous(), torch.zeros_like(k).contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, q_out=qo, k_out=ko, stream=side.cuda_stream)
    side.synchronize()
    close(qo, *plain(q, wq, pos, table, False), U[torch.bfloat16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.qk_norm_rope(q, k, pos, table, q_weight=wq, k_weight=wk, eps=EPS, q_out=qo, k_out=ko)
    pos.copy_((pos + 3) % 500)
    graph.replay()
    torch.cuda.synchronize()
    close(qo, *plain(q, wq, pos, table, False), U[torch.bfloat16])
    close(ko, *plain(k, wk, pos, table, False), U[torch.bfloat16])


def test_strides_of_single_elements_do_not_matter():
    q, k, v, pos, table, wq, wk = make(1, 3, 1, 64, 64, torch.bfloat16)
    odd = lambda t: t.contiguous().as_strided(t.shape, (1, 64 if t.shape[1] > 1 else 5, 1))  # noqa: E731
    kw = dict(q_weight=wq, k_weight=wk, eps=EPS)
    for a, b in zip(dg.qk_norm_rope(q, k, pos, table, **kw), dg.qk_norm_rope(odd(q), odd(k), pos, table, **kw)):
        assert torch.equal(a, b)
    for a, b in zip(dg.qk_norm_rope_backward(q, k, q, k, pos, table, **kw), dg.qk_norm_rope_backward(odd(q), odd(k), odd(q), odd(k), pos, table, **kw)):
        assert torch.equal(a, b)


def backward_case(tokens=300, seed=0):
    q, k, v, pos, table, wq, wk = make(tokens, 4, 2, 128, 128, torch.bfloat16, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    dq, dk = (torch.randn(t.shape, generator=gen, device="cuda").to(torch.bfloat16) for t in (q, k))
    return (dq, dk, q, k, pos, table), dict(q_weight=wq, k_weight=wk, eps=EPS)


def test_another_stream_than_the_current_one():
    """What is allocated for a call on another stream may not be memory that earlier work of the current stream still writes."""
    tensors, kw = backward_case()
    want = dg.qk_norm_rope_backward(*tensors, **kw)
    forward = dg.qk_norm_rope(*tensors[2:], **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in [512] * 8 + [1 << 20] * 3 + [1 << 19] * 3]
    torch.cuda._sleep(400_000_000)
    for t in freed:
        t.fill_(77)
    del freed, t
    got = dg.qk_norm_rope_backward(*tensors, stream=side.cuda_stream, **kw)
    rows = dg.qk_norm_rope(*tensors[2:], stream=side.cuda_stream, **kw)
    torch.cuda.synchronize()
    for a, b in zip(want + forward, got + rows):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):                        # from the side to the default stream, whose handle is 0
        got = dg.qk_norm_rope_backward(*tensors, stream=torch.cuda.default_stream().cuda_stream, **kw)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("explicit", [False, True])
def test_backward_in_a_graph(explicit):
    """A captured pass keeps scratch of its own: eager passes between replays change nothing; the stream may be given as well."""
    tensors, kw = backward_case()
    others, other_kw = backward_case(seed=5)
    want = dg.qk_norm_rope_backward(*tensors, **kw)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        if explicit:
            inner = torch.cuda.current_stream().cuda_stream
            with torch.cuda.stream(torch.cuda.Stream()):
                got = dg.qk_norm_rope_backward(*tensors, stream=inner, **kw)
        else:
            got = dg.qk_norm_rope_backward(*tensors, **kw)
    for _ in range(3):
        for t in got:
            t.zero_()
        dg.qk_norm_rope_backward(*others, **other_kw)
        graph.replay()
        dg.qk_norm_rope_backward(*others, **other_kw)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


def test_backward_from_several_threads():
    """Threads that share a stream: each pass is two launches, and another thread's may come between them."""
    cases = [backward_case(200 + 37 * i, seed=i) for i in range(4)]
    want = [dg.qk_norm_rope_backward(*t, **kw) for t, kw in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        t, kw = cases[i]
        for _ in range(40):
            got = dg.qk_norm_rope_backward(*t, **kw)
            if not all(torch.equal(a, b) for a, b in zip(want[i], got)):
                wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_refusals():
    q, k, v, pos, table, wq, wk = make(4, 2, 1, 64, 64, torch.bfloat16)
    for kw, err in ((dict(q=q.float()), TypeError), (dict(k=k.half()), TypeError), (dict(positions=pos.long()), TypeError),
                    (dict(table=table.double()), TypeError), (dict(q_weight=wq.float()), TypeError), (dict(q_weight=wq[:32]), ValueError),
                    (dict(positions=pos[:2]), ValueError), (dict(table=table.cpu()), ValueError), (dict(k=k[:2]), ValueError),
                    (dict(q=q.transpose(1, 2)), ValueError), (dict(q_weight=wq, norm=False), ValueError), (dict(v=v), ValueError)):
        args = dict(q=q, k=k, positions=pos, table=table)
        args.update(kw)
        with pytest.raises(err):
            dg.qk_norm_rope(args.pop("q"), args.pop("k"), args.pop("positions"), args.pop("table"), **args)
    with pytest.raises(dg.GemmError) as e:
        dg.qk_norm_rope(torch.zeros(4, 1, 20, dtype=torch.bfloat16, device="cuda"), None, pos, dg.rope_table(8, 8))
    assert e.value.status == dg.GEMM_ERR_UNSUPPORTED
    with pytest.raises(dg.GemmError) as e:                # rows 2 bytes off
        dg.qk_norm_rope(torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:257].view(4, 1, 64), None, pos, table)
    assert e.value.status == dg.GEMM_ERR_ALIGNMENT
    with pytest.raises(dg.GemmError) as e:                # wider than the head
        dg.qk_norm_rope(q, None, pos, dg.rope_table(8, 128))
    assert e.value.status == dg.GEMM_ERR_INVALID_ARG
