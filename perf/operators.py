"""The serving operators around the product, as cases with a plain form.

Three operators stand between the projections of an attention block:

  lora   Y = X W^T + s_i (X A_i^T) B_i^T, a shared projection and the low-rank adapter i of each token's request
  rope   RMS norm of every query and key head and its rotary position in one pass, into buffers or cache slots; its backward
  attn   attention of one new token per sequence over a paged key-value cache

``run`` computes them in elementary torch operations in 32 bits where ``own`` is false, and with this package's
kernels where it is true.  ``exact`` states the definitions again in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # four requests, one new token each, two adapters: the smallest call, where launches count
        dict(name="lora_decode_4", op="lora", tokens=4, requests=4, k=4096, n=4096, rank=16, adapters=2, type="bf16"),
        # a full decode batch in which nearly every request brings an adapter of its own
        dict(name="lora_decode_96", op="lora", tokens=96, requests=96, k=4096, n=4096, rank=16, adapters=80, type="bf16"),
        # odd sizes: ragged prompts of nine requests, rows and columns off every tile and alignment boundary
        dict(name="lora_odd_f16", op="lora", tokens=777, requests=9, k=1001, n=1543, rank=24, adapters=5, type="f16"),
        # prompts of twelve requests through a square projection: the library's largest matrix size
        dict(name="lora_prefill_8192", op="lora", tokens=8192, requests=12, k=8192, n=8192, rank=64, adapters=8, type="bf16"),
        # one decode step's tokens: queries out, keys and values into their cache slots
        dict(name="rope_decode_16", op="rope", dir="cache", tokens=16, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             weights=True, page=16, positions=32768, type="bf16", cache="bf16"),
        # part of an odd-sized head rotated in pairs, no norm weights, an 8-bit cache of odd pages
        dict(name="rope_partial_e4m3", op="rope", dir="cache", tokens=1231, heads=12, kv_heads=3, dim=80, rot=32, layout="pairs",
             weights=False, page=24, positions=8192, type="f16", cache="e4m3"),
        # a long prompt's queries, keys and values
        dict(name="rope_prefill_16384", op="rope", dir="cache", tokens=16384, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             weights=True, page=16, positions=131072, type="bf16", cache="bf16"),
        # the backward pass of a training batch
        dict(name="rope_backward_8192", op="rope", dir="backward", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             weights=True, page=16, positions=8192, type="bf16", cache="bf16"),
        # one short sequence: the smallest call
        dict(name="attn_short_1", op="attn", batch=1, low=150, high=150, kv_heads=8, group=4, dim=64, page=16, window=0, type="bf16", cache="bf16"),
        # a decode batch of ragged lengths, one of them empty, up to 8192 tokens
        dict(name="attn_ragged_64", op="attn", batch=64, low=0, high=8192, kv_heads=8, group=4, dim=128, page=16, window=0, type="bf16", cache="bf16"),
        # an 8-bit cache seen through a sliding window, odd group and head sizes
        dict(name="attn_window_e4m3", op="attn", batch=33, low=700, high=9001, kv_heads=4, group=7, dim=80, page=24, window=2001, type="f16", cache="e4m3"),
        # two long contexts: work has to be split over the cache's length
        dict(name="attn_long_131072", op="attn", batch=2, low=130001, high=131072, kv_heads=8, group=8, dim=128, page=64, window=0, type="bf16", cache="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lora", "rope", "attn"))
    kind = rng.choice(("bf16", "f16"))
    if op == "lora":
        tokens = _log(rng, 1, 8192)
        adapters = _log(rng, 1, 64)
        return dict(op="lora", tokens=tokens, requests=min(tokens, _log(rng, 1, 128)), k=_log(rng, 256, 8192), n=_log(rng, 256, 8192),
                    rank=rng.choice((8, 16, 24, 32, 64)), adapters=adapters, type=kind)
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 256))
        kv = rng.choice((1, 2, 4, 8))
        return dict(op="rope", dir=rng.choice(("cache", "plain", "backward")), tokens=_log(rng, 1, 8192), heads=kv * rng.choice((1, 2, 3, 4)),
                    kv_heads=kv, dim=dim, rot=rng.choice((dim, dim // 2, 32, 24)), layout=rng.choice(("half", "pairs")),
                    weights=rng.random() < 0.7, page=rng.choice((1, 8, 16, 24, 64)), positions=32768, type=kind,
                    cache=rng.choice((kind, "e4m3")))
    dim = rng.choice((64, 80, 96, 128, 256))
    kv = rng.choice((1, 2, 4, 8))
    batch = _log(rng, 1, 128)
    high = _log(rng, 1, min(131072, (1 << 27) // (batch * kv * dim)))
    return dict(op="attn", batch=batch, low=rng.randint(0, high), high=high, kv_heads=kv, group=rng.choice((1, 2, 3, 4, 5, 7, 8, 16)), dim=dim,
                page=rng.choice((1, 8, 16, 24, 32, 64)), window=rng.choice((0, 0, max(1, high // 3))), type=kind, cache=rng.choice((kind, "e4m3")))


# ---------------------------------------------------------------- sizes that follow from a case alone

def _lengths(c):
    """Lengths of an attention case's sequences: from low to high, evenly over their logarithm."""
    lo, hi, n = c["low"], c["high"], c["batch"]
    if n == 1:
        return [hi]
    rest = [round(math.exp(math.log(max(lo, 1)) + (math.log(max(hi, 1)) - math.log(max(lo, 1))) * i / (n - 1))) for i in range(n)]
    rest[-1] = hi
    rest[0] = lo
    return rest


def _request_lengths(tokens, requests):
    """Ragged request lengths that add up to `tokens`, the later ones longer."""
    if requests == tokens:
        return [1] * tokens
    total = requests * (requests + 1) // 2
    cut = [tokens * (i * (i + 1) // 2) // total for i in range(requests + 1)]
    return [b - a for a, b in zip(cut, cut[1:])]


def work(case):
    c = case
    if c["op"] == "lora":
        m, k, n, r = c["tokens"], c["k"], c["n"], c["rank"]
        used = min(c["adapters"], c["requests"])
        return {"bytes": 2.0 * (m * k + n * k + m * n + used * r * (k + n)) + 4.0 * m,
                "flops": 2.0 * m * n * k + 2.0 * m * r * (k + n)}
    if c["op"] == "rope":
        t, d, rows = c["tokens"], c["dim"], c["tokens"] * (c["heads"] + c["kv_heads"])
        table = 4.0 * t * c["rot"] + 4.0 * t
        if c["dir"] == "backward":
            return {"bytes": 3 * 2.0 * rows * d + table, "flops": 14.0 * rows * d}
        e = BYTES[c["cache"]] if c["dir"] == "cache" else 2
        kv = t * c["kv_heads"] * d
        data = 2.0 * rows * d + 2.0 * t * c["heads"] * d + e * kv
        if c["dir"] == "cache":
            data += (2.0 + e) * kv + 4.0 * t
        return {"bytes": data + table, "flops": 8.0 * rows * d}
    seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    heads = c["kv_heads"] * c["group"]
    return {"bytes": 2.0 * BYTES[c["cache"]] * seen * c["kv_heads"] * c["dim"] + 4.0 * c["batch"] * heads * c["dim"],
            "flops": 4.0 * seen * heads * c["dim"]}


# ---------------------------------------------------------------- inputs

def _padded(rows, cols, gen, kind, scale=1.0):
    """A [rows, cols] matrix whose rows start on 16-byte boundaries, as an allocator of activations pads them."""
    ld = -(-cols // 8) * 8
    return (torch.randn(rows, ld, generator=gen, device="cuda") * scale).to(TYPES[kind])[:, :cols]


def _table(positions, rot, base=10000.0):
    """cos and sin of position x base^(-2i/rot), [positions, 2, rot / 2] in 32 bits."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack((a.cos(), a.sin()), 1).float().contiguous()


def _prepare_lora(c, gen):
    m, k, n, r, count = c["tokens"], c["k"], c["n"], c["rank"], c["adapters"]
    kind = c["type"]
    s = dict(x=_padded(m, k, gen, kind), w=_padded(n, k, gen, kind, k ** -0.5))
    s["a"] = _padded(count * r, k, gen, kind, k ** -0.5).unflatten(0, (count, r))
    s["b"] = (torch.randn(count, n, r, generator=gen, device="cuda") * 0.3).to(TYPES[kind])
    s["scale"] = 0.5 + torch.rand(count, generator=gen, device="cuda")
    # requests take the adapters in turn, every (count + 1)-th one none; which comes where goes by the seed
    ids = torch.arange(c["requests"], device="cuda") % (count + 1)
    ids = torch.where(ids == count, -1, ids)[torch.randperm(c["requests"], generator=gen, device="cuda")]
    lengths = torch.tensor(_request_lengths(m, c["requests"]), device="cuda")
    s["adapter"] = ids.repeat_interleave(lengths).to(torch.int32)
    s["y"] = torch.empty(m, -(-n // 8) * 8, dtype=TYPES[kind], device="cuda")[:, :n]
    if own:
        import dense_gemm_blackwell_gb300 as dg
        s["plan"] = dg.LoraPlan(m, n, k, rank=r, adapters=count, dtype=dg.GEMM_BF16 if kind == "bf16" else dg.GEMM_F16,
                                ldx=s["x"].stride(0), ldw=s["w"].stride(0), ldy=s["y"].stride(0))
    return s


def _prepare_rope(c, gen):
    t, h, g, d, rot = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    kind = TYPES[c["type"]]
    # one projection's output: queries, keys and values side by side
    qkv = torch.randn(t, (h + 2 * g) * d, generator=gen, device="cuda").to(kind)
    s = dict(q=qkv[:, : h * d].unflatten(1, (h, d)), k=qkv[:, h * d: (h + g) * d].unflatten(1, (g, d)), v=qkv[:, (h + g) * d:].unflatten(1, (g, d)))
    s["positions"] = torch.randint(0, c["positions"], (t,), generator=gen, device="cuda").to(torch.int32)
    s["table"] = _table(c["positions"], rot)
    s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(kind) if c["weights"] else None
    s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(kind) if c["weights"] else None
    s["interleaved"] = c["layout"] == "pairs"
    s["q_out"] = torch.empty(t, h, d, dtype=kind, device="cuda")
    if c["dir"] == "cache":
        pages = -(-t // c["page"]) + 3
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = (order[at // c["page"]] * c["page"] + at % c["page"]).to(torch.int32)
        s["k_cache"] = torch.zeros(pages, c["page"], g, d, device="cuda").to(TYPES[c["cache"]])
        s["v_cache"] = torch.zeros(pages, c["page"], g, d, device="cuda").to(TYPES[c["cache"]])
        s["k_scale"], s["v_scale"] = (0.03125, 0.02) if c["cache"] == "e4m3" else (1.0, 1.0)
    else:
        s["k_out"] = torch.empty(t, g, d, dtype=kind, device="cuda")
    if c["dir"] == "backward":
        s["dq"] = torch.randn(t, h, d, generator=gen, device="cuda").to(kind)
        s["dk"] = torch.randn(t, g, d, generator=gen, device="cuda").to(kind)
    return s


def _prepare_attn(c, gen):
    b, g, d, page = c["batch"], c["kv_heads"], c["dim"], c["page"]
    kind, cache = TYPES[c["type"]], TYPES[c["cache"]]
    lengths = torch.tensor(_lengths(c), device="cuda")[torch.randperm(b, generator=gen, device="cuda")]
    width = max(1, -(-c["high"] // page))
    used = -(-lengths // page)
    pages = int(sum(-(-n // page) for n in _lengths(c))) + 2
    # a cache in use: every sequence's pages lie scattered over it
    order = torch.randperm(pages, generator=gen, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    at = (used.cumsum(0) - used)[:, None] + col
    table = torch.where(col < used[:, None], order[at.clamp(max=pages - 1)], -1).to(torch.int32)
    s = dict(q=torch.randn(b, g * c["group"], d, generator=gen, device="cuda").to(kind), lengths=lengths.to(torch.int32), block_table=table)
    s["k_scale"], s["v_scale"] = (0.03125, 0.02) if c["cache"] == "e4m3" else (1.0, 1.0)
    s["k_cache"] = (torch.randn(pages, page, g, d, generator=gen, device="cuda") / s["k_scale"]).to(cache)
    s["v_cache"] = (torch.randn(pages, page, g, d, generator=gen, device="cuda") / s["v_scale"]).to(cache)
    s["softmax_scale"] = d ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b, g * c["group"], dtype=torch.float32, device="cuda")
    if own:
        import dense_gemm_blackwell_gb300 as dg
        codes = {"bf16": dg.GEMM_BF16, "f16": dg.GEMM_F16, "e4m3": dg.GEMM_E4M3}
        s["plan"] = dg.PagedAttentionPlan(b, heads=g * c["group"], kv_heads=g, head_dim=d, page_size=page, dtype=codes[c["type"]],
                                          dtype_cache=codes[c["cache"]], window=c["window"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = {"lora": _prepare_lora, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]]
    return dict(make(case, gen), case=case)


# ---------------------------------------------------------------- the plain forms

def _plain_lora(s):
    a, b = s["a"].float(), s["b"].float()
    count, r = a.shape[:2]
    x = s["x"].float()
    mine = s["adapter"][:, None] == torch.arange(count, device=x.device)
    t = (x @ a.flatten(0, 1).T).unflatten(1, (count, r)) * (mine * s["scale"])[:, :, None]
    s["y"].copy_(x @ s["w"].float().T + t.flatten(1) @ b.transpose(1, 2).flatten(0, 1))
    return s["y"]


def _split(y, rot, interleaved):
    part = y[..., :rot]
    return (part[..., 0::2], part[..., 1::2]) if interleaved else part.chunk(2, -1)


def _join(a, b, rest, interleaved):
    part = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((part, rest), -1)


def _turn(y, cos, sin, rot, interleaved):
    a, b = _split(y, rot, interleaved)
    return _join(a * cos - b * sin, a * sin + b * cos, y[..., rot:], interleaved)


def _plain_norm(x, weight):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return n if weight is None else n * weight.float()


def _store(cache, slots, rows, scale):
    """Rows into their slots of the cache, rounded once."""
    if cache.dtype == torch.float8_e4m3fn:
        rows = (rows / scale).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)
        cache.view(torch.uint8).flatten(0, 1)[slots] = rows.view(torch.uint8)
    else:
        cache.flatten(0, 1)[slots] = rows.to(cache.dtype)


def _plain_rope(s):
    c = s["case"]
    cos, sin = s["table"][s["positions"].long()].unbind(1)
    cos, sin, rot, pairs = cos[:, None], sin[:, None], c["rot"], s["interleaved"]
    if c["dir"] == "backward":
        return _plain_rope_backward(s["q"], s["dq"], s["q_weight"], cos, sin, rot, pairs) + _plain_rope_backward(
            s["k"], s["dk"], s["k_weight"], cos, sin, rot, pairs)
    s["q_out"].copy_(_turn(_plain_norm(s["q"].float(), s["q_weight"]), cos, sin, rot, pairs))
    k = _turn(_plain_norm(s["k"].float(), s["k_weight"]), cos, sin, rot, pairs)
    if c["dir"] == "plain":
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    slots = s["slots"].long()
    _store(s["k_cache"], slots, k, s["k_scale"])
    _store(s["v_cache"], slots, s["v"].float(), s["v_scale"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_rope_backward(x, dy, weight, cos, sin, rot, pairs):
    kind = x.dtype
    x = x.float()
    g = _turn(dy.float(), cos, -sin, rot, pairs)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    if weight is None:
        return ((r * (g - n * (g * n).mean(-1, keepdim=True))).to(kind),)
    gw = g * weight.float()
    return (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(kind), (g * n).sum((0, 1))


def _plain_attn(s):
    c = s["case"]
    b, heads, d = s["q"].shape
    g = c["kv_heads"]
    table = s["block_table"].clamp(min=0).long()
    k, v = (s[n + "_cache"][table].flatten(1, 2).float() * s[n + "_scale"] for n in "kv")
    q = s["q"].float().unflatten(1, (g, heads // g)) * s["softmax_scale"]
    score = q @ k.permute(0, 2, 3, 1)
    at = torch.arange(k.shape[1], device=q.device)
    lengths = s["lengths"].long()[:, None]
    seen = at < lengths
    if c["window"]:
        seen &= at >= lengths - c["window"]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = v.permute(0, 2, 1, 3).masked_fill(~seen[:, None, :, None], 0.0)
    s["out"].copy_(((p @ v) / total.clamp(min=1e-30)).flatten(1, 2))
    s["lse"].copy_(torch.where(total > 0, top + total.log(), -math.inf).flatten(1))
    return s["out"], s["lse"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"lora": _plain_lora, "rope": _plain_rope, "attn": _plain_attn}[c["op"]](s)
    import dense_gemm_blackwell_gb300 as dg
    if c["op"] == "lora":
        s["plan"].run(s["x"], s["w"], s["a"], s["b"], s["adapter"], s["y"], scale=s["scale"])
        return s["y"]
    if c["op"] == "attn":
        s["plan"].run(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lengths"], s["out"], lse=s["lse"], scale=s["softmax_scale"],
                      k_scale=s["k_scale"], v_scale=s["v_scale"])
        return s["out"], s["lse"]
    norm = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"])
    if c["dir"] == "backward":
        dq, dk, dqw, dkw = dg.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["table"], dq_out=s["q_out"],
                                                    dk_out=s["k_out"], **norm)
        return (dq, dqw, dk, dkw) if c["weights"] else (dq, dk)
    if c["dir"] == "plain":
        return dg.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], q_out=s["q_out"], k_out=s["k_out"], **norm)
    dg.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], q_out=s["q_out"], v=s["v"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                    slots=s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"], **norm)
    return s["q_out"], s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_lora(s):
    x = s["x"].double()
    y = x @ s["w"].double().T
    for i in range(s["a"].shape[0]):
        rows = (s["adapter"] == i).nonzero().flatten()
        y[rows] += float(s["scale"][i]) * ((x[rows] @ s["a"][i].double().T) @ s["b"][i].double().T)
    return y


def _exact_turn(x, weight, s, rot):
    n = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    if weight is not None:
        n = n * weight.double()
    angle = s["table"].double()[s["positions"].long()]
    first = torch.arange(0, rot, 2, device=x.device) if s["interleaved"] else torch.arange(rot // 2, device=x.device)
    second = first + (1 if s["interleaved"] else rot // 2)
    z = torch.complex(n[..., first], n[..., second]) * torch.complex(angle[:, 0], angle[:, 1])[:, None]
    out = n.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(s):
    c = s["case"]
    rot = c["rot"]
    if c["dir"] == "backward":
        found = []
        for x, dy, weight in ((s["q"], s["dq"], s["q_weight"]), (s["k"], s["dk"], s["k_weight"])):
            inputs = [x.double().requires_grad_()] + ([weight.double().requires_grad_()] if weight is not None else [])
            out = _exact_turn(inputs[0], inputs[1] if weight is not None else None, s, rot)
            found += list(torch.autograd.grad(out, inputs, dy.double()))
        return tuple(found)
    q, k = _exact_turn(s["q"].double(), s["q_weight"], s, rot), _exact_turn(s["k"].double(), s["k_weight"], s, rot)
    if c["dir"] == "plain":
        return q, k
    caches = []
    for cache, rows, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        full = cache.double()
        full.flatten(0, 1)[s["slots"].long()] = (rows / scale).clamp(-E4M3_MAX, E4M3_MAX) if c["cache"] == "e4m3" else rows
        caches.append(full)
    return q, caches[0], caches[1]


def _exact_attn(s):
    c = s["case"]
    b, heads, d = s["q"].shape
    g, page = c["kv_heads"], c["page"]
    out = torch.zeros(b, heads, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, heads), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        pages = s["block_table"][i, : -(-n // page)].long()
        for h in range(g):
            k = s["k_cache"][pages, :, h].reshape(-1, d)[first:n].double() * s["k_scale"]
            v = s["v_cache"][pages, :, h].reshape(-1, d)[first:n].double() * s["v_scale"]
            mine = slice(h * (heads // g), (h + 1) * (heads // g))
            score = (s["q"][i, mine].double() @ k.T) * s["softmax_scale"]
            lse[i, mine] = torch.logsumexp(score, -1)
            out[i, mine] = torch.softmax(score, -1) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"lora": _exact_lora, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](s)
