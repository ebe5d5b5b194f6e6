"""The operators of a feed-forward block, as cases with a plain form.

Three operators make up the block that follows attention in a layer:

  norm   the residual's addition and its RMS norm in one pass, in 16 bits or as E4M3 codes with the scales that the
         products read; its backward pass
  gated  act(X Wg^T) * (X Wu^T), both projections, the activation and the product in one kernel; its backward pass
  int4   products of a few tokens with 4-bit weights and group scales, alone or as a gated pair of projections

``run`` computes them in elementary torch operations in 32 bits where ``own`` is false, and with this package's
kernels where it is true.  ``exact`` states the definitions again in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -100
EPS = 1e-6


def listed():
    return [
        # one decode step of eight requests: the smallest call, where launches count
        dict(name="norm_decode_8", op="norm", dir="forward", tokens=8, hidden=4096, out="same", residual=True, weight=True, type="bf16"),
        # odd sizes: rows that end inside a vector, a scale block and a tile of scales
        dict(name="norm_mx_odd_f16", op="norm", dir="forward", tokens=1231, hidden=2893, out="mx", residual=True, weight=True, type="f16"),
        # a long prompt's rows into the block-scaled product of the library's largest square size
        dict(name="norm_prefill_8192", op="norm", dir="forward", tokens=8192, hidden=8192, out="block128", residual=True, weight=True, type="bf16"),
        # the backward pass of a training batch
        dict(name="norm_backward_8192", op="norm", dir="backward", tokens=8192, hidden=4096, out="same", residual=True, weight=True, type="bf16"),
        # four requests, one new token each: the time is the stream of the weights
        dict(name="gated_decode_4", op="gated", dir="forward", tokens=4, k=4096, features=12288, act="silu", type="bf16"),
        # a full decode batch
        dict(name="gated_decode_96", op="gated", dir="forward", tokens=96, k=4096, features=12288, act="silu", type="bf16"),
        # odd sizes: ragged prompts, rows and columns off every tile
        dict(name="gated_odd_f16", op="gated", dir="forward", tokens=777, k=1001, features=1544, act="gelu", type="f16"),
        # prompts of several requests
        dict(name="gated_prefill_8192", op="gated", dir="forward", tokens=8192, k=4096, features=16384, act="silu", type="bf16"),
        # the gradients of a training batch: of the rows and of both weights
        dict(name="gated_backward_4096", op="gated", dir="backward", tokens=4096, k=4096, features=8192, act="silu", type="bf16"),
        # one new token through a square projection
        dict(name="int4_decode_1", op="int4", tokens=1, k=4096, n=4096, group=128, zeros=False, act="", type="bf16"),
        # eight requests through the gated pair of projections, zero points of every group
        dict(name="int4_gated_8", op="int4", tokens=8, k=4096, n=24576, group=128, zeros=True, act="silu", type="bf16"),
        # odd numbers of tokens and outputs, small groups, the last of them cut short
        dict(name="int4_odd_f16", op="int4", tokens=13, k=5130, n=1543, group=32, zeros=True, act="", type="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "gated", "int4"))
    kind = rng.choice(("bf16", "f16"))
    if op == "norm":
        hidden = _log(rng, 128, 16384)
        back = rng.random() < 0.35
        return dict(op="norm", dir="backward" if back else "forward", tokens=_log(rng, 1, min(16384, (1 << 25) // hidden)), hidden=hidden,
                    out="same" if back else rng.choice(("same", "block128", "mx")), residual=rng.random() < 0.7, weight=rng.random() < 0.8, type=kind)
    if op == "gated":
        back = rng.random() < 0.4
        return dict(op="gated", dir="backward" if back else "forward", tokens=_log(rng, 1, 2048 if back else 4096), k=_log(rng, 256, 4096),
                    features=8 * _log(rng, 32, 1024 if back else 1536), act=rng.choice(("silu", "gelu", "gelu_tanh")), type=kind)
    act = rng.choice(("", "silu", "gelu"))
    return dict(op="int4", tokens=rng.randint(1, 16), k=2 * _log(rng, 128, 6144), n=(2 if act else 1) * _log(rng, 200, 8192),
                group=rng.choice((32, 64, 96, 128, 256)), zeros=rng.random() < 0.6, act=act, type=kind)


def work(case):
    c = case
    if c["op"] == "norm":
        t, n = c["tokens"], c["hidden"]
        weight = 2.0 * n if c["weight"] else 0.0
        if c["dir"] == "backward":
            return {"bytes": (8.0 if c["residual"] else 6.0) * t * n + (weight and weight + 4.0 * n), "flops": 11.0 * t * n}
        y = {"same": 2.0 * n, "block128": n + 4.0 * -(-n // 128), "mx": n + 1.0 * -(-n // 32)}[c["out"]]
        return {"bytes": t * ((6.0 if c["residual"] else 2.0) * n + y) + weight, "flops": 6.0 * t * n}
    if c["op"] == "gated":
        t, k, f = c["tokens"], c["k"], c["features"]
        if c["dir"] == "backward":
            return {"bytes": 2.0 * (3 * t * f + 2 * t * k + 4 * f * k), "flops": 8.0 * t * f * k + 16.0 * t * f}
        return {"bytes": 2.0 * (t * k + 2 * f * k + t * f), "flops": 4.0 * t * f * k + 8.0 * t * f}
    t, k, n, groups = c["tokens"], c["k"], c["n"], -(-c["k"] // c["group"])
    return {"bytes": n * k / 2 + (3.0 if c["zeros"] else 2.0) * n * groups + 2.0 * t * (k + (n // 2 if c["act"] else n)), "flops": 2.0 * t * n * k}


# ---------------------------------------------------------------- inputs

def _padded(rows, cols, gen, kind, scale=1.0):
    """A [rows, cols] matrix whose rows start on 16-byte boundaries, as an allocator of activations pads them."""
    ld = -(-cols // 8) * 8
    return (torch.randn(rows, ld, generator=gen, device="cuda") * scale).to(TYPES[kind])[:, :cols]


def _rows(rows, cols, dtype, to=8):
    """Room for [rows, cols] in rows of a multiple of `to` elements."""
    return torch.zeros(rows, -(-cols // to) * to, device="cuda").to(dtype)[:, :cols]


def _prepare_norm(c, gen):
    t, n, kind = c["tokens"], c["hidden"], c["type"]
    s = dict(weight=(1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(TYPES[kind]) if c["weight"] else None)
    if c["dir"] == "backward":
        # the sum that the forward pass left, the gradient of its norm and, with a residual, the one that comes along it
        s.update(h=_padded(t, n, gen, kind, 2.0), dy=_padded(t, n, gen, kind), dh=_rows(t, n, TYPES[kind]))
        s["dsum"] = _padded(t, n, gen, kind) if c["residual"] else None
        return s
    s.update(x=_padded(t, n, gen, kind), residual=_padded(t, n, gen, kind, 2.0) if c["residual"] else None)
    s["h"] = _rows(t, n, TYPES[kind]) if c["residual"] else None
    if c["out"] == "same":
        s["y"] = _rows(t, n, TYPES[kind])
    else:
        s["y"] = _rows(t, n, torch.float8_e4m3fn, 16)
        if c["out"] == "block128":
            s["scales"] = torch.zeros(t, -(-n // 128), device="cuda")
        else:
            s["scales"] = torch.zeros(-(-t // 128) * -(-n // 128) * 512, dtype=torch.uint8, device="cuda")
    return s


def _prepare_gated(c, gen):
    t, k, f, kind = c["tokens"], c["k"], c["features"], c["type"]
    s = dict(x=_padded(t, k, gen, kind), w=_padded(2 * f, k, gen, kind, 1.5 * k ** -0.5))
    if c["dir"] == "forward":
        s["h"] = _rows(t, f, TYPES[kind])
    else:
        # what the forward pass kept: both projections, rounded
        s["gate_up"] = (s["x"].float() @ s["w"].float().T).to(TYPES[kind])
        s["dh"] = _padded(t, f, gen, kind)
        s["dx"], s["dw"] = _rows(t, k, TYPES[kind]), _rows(2 * f, k, TYPES[kind])
    if own:
        import dense_gemm_blackwell_gb300 as dg
        s["plan"] = dg.GatedPlan(t, f, k, activation=c["act"], dtype=dg.GEMM_BF16 if kind == "bf16" else dg.GEMM_F16, ldx=s["x"].stride(0),
                                 ldw=s["w"].stride(0), gradients=c["dir"] == "backward")
    return s


def _prepare_int4(c, gen):
    t, k, n, kind = c["tokens"], c["k"], c["n"], c["type"]
    groups = -(-k // c["group"])
    s = dict(x=_padded(t, k, gen, kind))
    # two codes a byte, the even one in the low half
    s["codes"] = torch.randint(0, 256, (n, -(-k // 32) * 16), generator=gen, device="cuda").to(torch.uint8)[:, : k // 2]
    s["scales"] = ((0.5 + torch.rand(n, groups, generator=gen, device="cuda")) * 0.25 * k ** -0.5).to(TYPES[kind])
    s["zeros"] = torch.randint(5, 11, (n, groups), generator=gen, device="cuda").to(torch.uint8) if c["zeros"] else None
    s["y"] = torch.empty(t, n // 2 if c["act"] else n, dtype=TYPES[kind], device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    make = {"norm": _prepare_norm, "gated": _prepare_gated, "int4": _prepare_int4}[case["op"]]
    return dict(make(case, gen), case=case)


# ---------------------------------------------------------------- the plain forms

def _blocks(n, size, v):
    """v [rows, n] cut into blocks of `size` columns, the last one filled up with zeros: [rows, blocks, size]."""
    return torch.nn.functional.pad(v, (0, -n % size)).unflatten(1, (-1, size))


def _tiled(bytes_, rows, cols):
    """[rows, cols] scale bytes as 512-byte tiles of 128 rows x 4 columns, byte (r mod 32) 16 + (r / 32 mod 4) 4 + c mod 4."""
    full = torch.nn.functional.pad(bytes_, (0, -cols % 4, 0, -rows % 128))
    return full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _plain_norm(s):
    c = s["case"]
    t, n = c["tokens"], c["hidden"]
    if c["dir"] == "backward":
        h, g = s["h"].float(), s["dy"].float()
        r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        unit = h * r
        gw = g if s["weight"] is None else g * s["weight"].float()
        dh = r * (gw - unit * (gw * unit).mean(1, keepdim=True))
        s["dh"].copy_(dh if s["dsum"] is None else dh + s["dsum"].float())
        return (s["dh"],) if s["weight"] is None else (s["dh"], (g * unit).sum(0))
    h = s["x"].float()
    kept = ()
    if s["residual"] is not None:
        s["h"].copy_(h + s["residual"].float())
        h, kept = s["h"].float(), (s["h"],)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if c["out"] == "same":
        s["y"].copy_(y)
        return (s["y"],) + kept
    if c["out"] == "block128":
        blocks = _blocks(n, 128, y)
        scale = (blocks.abs().amax(2) / E4M3_MAX).clamp(min=LEAST_SCALE)
        s["scales"].copy_(scale)
        scales = s["scales"]
    else:
        blocks = _blocks(n, 32, y)
        # the least power of two that keeps the block within the type's range
        half, power = torch.frexp(blocks.abs().amax(2))
        power = torch.where(half > 0.875, power - 8, power - 9)
        power = torch.where(half == 0, -126, power).clamp(-126, 127) + 127
        s["scales"].copy_(_tiled(power.to(torch.uint8), t, power.shape[1]))
        scale, scales = (power << 23).view(torch.float32), s["scales"].view(torch.float8_e8m0fnu)
    codes = (blocks / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(1)[:, :n].to(torch.float8_e4m3fn)
    s["y"].copy_(codes)
    return (s["y"], scales) + kept


def _plain_act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))
    return 0.5 * g * (1 + torch.tanh((2 / math.pi) ** 0.5 * (g + 0.044715 * g * g * g)))


def _plain_slope(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * 0.5 ** 0.5)) + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    a = (2 / math.pi) ** 0.5
    th = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * a * (1 + 3 * 0.044715 * g * g)


def _plain_gated(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    if c["dir"] == "forward":
        gate, up = (x @ w.T).chunk(2, 1)
        s["h"].copy_(_plain_act(gate, c["act"]) * up)
        return s["h"]
    gate, up = s["gate_up"].float().chunk(2, 1)
    dh = s["dh"].float()
    both = torch.cat((dh * up * _plain_slope(gate, c["act"]), dh * _plain_act(gate, c["act"])), 1)
    s["dx"].copy_(both @ w)
    s["dw"].copy_(both.T @ x)
    return s["dx"], s["dw"]


def _plain_int4(s):
    c = s["case"]
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).flatten(1).float()
    blocks = _blocks(c["k"], c["group"], codes)
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, :, None]
    w = ((blocks - zero) * s["scales"].float()[:, :, None]).flatten(1)[:, : c["k"]]
    y = s["x"].float() @ w.T
    if c["act"]:
        gate, up = y.chunk(2, 1)
        y = _plain_act(gate, c["act"]) * up
    s["y"].copy_(y)
    return s["y"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "gated": _plain_gated, "int4": _plain_int4}[c["op"]](s)
    import dense_gemm_blackwell_gb300 as dg
    if c["op"] == "int4":
        return dg.int4_matmul(s["x"], s["codes"], s["scales"], group=c["group"], zeros=s["zeros"], activation=c["act"] or None, out=s["y"])
    if c["op"] == "gated":
        if c["dir"] == "forward":
            return s["plan"].run(s["x"], s["w"], s["h"])
        return s["plan"].backward(s["dh"], s["x"], s["w"], s["gate_up"], s["dx"], s["dw"])
    if c["dir"] == "backward":
        dh, dweight = dg.add_rms_norm_backward(s["dy"], s["h"], s["weight"], d_sum=s["dsum"], eps=EPS, out=s["dh"])
        return (dh,) if dweight is None else (dh, dweight)
    mode = {"same": dg.GEMM_SCALE_NONE, "block128": dg.GEMM_SCALE_BLOCK_1x128_128x128, "mx": dg.GEMM_SCALE_MX_E8M0_32}[c["out"]]
    y, scales, h = dg.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, out=s["y"], sum_out=s["h"], scale_mode=mode,
                                   scales=s.get("scales"))
    if c["out"] == "mx":
        scales = scales.view(torch.float8_e8m0fnu)
    return tuple(v for v in (y, scales, h) if v is not None)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(s):
    c = s["case"]
    t, n = c["tokens"], c["hidden"]

    def normed(h, weight):
        y = h / (h.pow(2).mean(1, keepdim=True) + EPS).sqrt()
        return y if weight is None else y * weight

    if c["dir"] == "backward":
        inputs = [s["h"].double().requires_grad_()] + ([] if s["weight"] is None else [s["weight"].double().requires_grad_()])
        found = list(torch.autograd.grad(normed(inputs[0], inputs[1] if len(inputs) > 1 else None), inputs, s["dy"].double()))
        if s["dsum"] is not None:
            found[0] = found[0] + s["dsum"].double()
        return tuple(found)
    h, kept = s["x"].double(), ()
    if s["residual"] is not None:
        h = h + s["residual"].double()
        kept = (h,)
        h = h.to(s["x"].dtype).double()        # the norm is that of the sum as it is kept
    y = normed(h, None if s["weight"] is None else s["weight"].double())
    if c["out"] == "same":
        return (y,) + kept
    size = 128 if c["out"] == "block128" else 32
    columns = -(-n // size)
    top = torch.zeros(t, columns, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, (torch.arange(n, device="cuda") // size).expand(t, n), y.abs(), "amax")
    if c["out"] == "block128":
        scale = (top / E4M3_MAX).clamp(min=LEAST_SCALE)
        given = scale
    else:
        scale = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=-126.0))
        r, q = torch.arange(t, device="cuda")[:, None], torch.arange(columns, device="cuda")[None, :]
        wide = -(-columns // 4)
        given = torch.full((-(-t // 128) * wide * 512,), 2.0 ** -127, dtype=torch.float64, device="cuda")
        given[(r // 128 * wide + q // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + q % 4] = scale
    return (y / scale.repeat_interleave(size, 1)[:, :n], given) + kept


def _exact_act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return torch.nn.functional.gelu(g, approximate="tanh" if act == "gelu_tanh" else "none")


def _exact_gated(s):
    c = s["case"]
    x, w, f = s["x"].double(), s["w"].double(), c["features"]
    if c["dir"] == "forward":
        return _exact_act(x @ w[:f].T, c["act"]) * (x @ w[f:].T)
    gate, up = (s["gate_up"][:, i * f: (i + 1) * f].double().requires_grad_() for i in (0, 1))
    dgate, dup = torch.autograd.grad(_exact_act(gate, c["act"]) * up, (gate, up), s["dh"].double())
    return dgate @ w[:f] + dup @ w[f:], torch.cat((dgate.T @ x, dup.T @ x))


def _exact_int4(s):
    c = s["case"]
    k, group = c["k"], c["group"]
    w = torch.empty(c["n"], k, dtype=torch.float64, device="cuda")
    w[:, 0::2] = s["codes"].remainder(16).double()
    w[:, 1::2] = s["codes"].div(16, rounding_mode="floor").double()
    at = torch.arange(k, device="cuda") // group
    w = (w - (8.0 if s["zeros"] is None else s["zeros"].double()[:, at])) * s["scales"].double()[:, at]
    x = s["x"].double()
    if not c["act"]:
        return x @ w.T
    half = c["n"] // 2
    return _exact_act(x @ w[:half].T, c["act"]) * (x @ w[half:].T)


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "gated": _exact_gated, "int4": _exact_int4}[case["op"]](s)
