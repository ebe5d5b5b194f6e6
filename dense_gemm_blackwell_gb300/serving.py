"""Operators that stand between the products of an attention block (include/serving.h).

* :class:`LoraPlan`, :func:`lora_matmul`: a shared projection with the low-rank adapter of each token's request.
* :func:`qk_norm_rope`, :func:`qk_norm_rope_backward`: RMS norm of query and key heads with their rotary positions in one
  pass, optionally into a paged key-value cache; :func:`rope_table` makes the cosines and sines.
* :class:`PagedAttentionPlan`: attention of one new token per sequence over that cache.

As in the rest of the package this is argument marshalling: shapes, types, strides and devices are checked here, the
work is enqueued by the CUDA library on torch's current stream (or the one given), and errors raise GemmError (from the
library) or ValueError / TypeError (from these checks).  Outputs that are not given, and scratch memory, are allocated by
torch for the stream that the work goes to.  A plan's launches share its workspace, so launches of one plan (and graphs
that captured it) must follow one another.  None of these calls enters torch's autograd graph: training calls
qk_norm_rope_backward itself, from an autograd function of its own for instance.
"""
from __future__ import annotations

import ctypes
import itertools
import math
import os
import re
import threading

from . import (GEMM_BF16, GEMM_E4M3, GEMM_F16, GEMM_F32, GEMM_OK, GemmDeviceError, GemmError, GemmPlanInfo, _dtype_code,
               current_stream_handle, lib)

SERVING_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "serving.h")
_I32, _I64, _F32, _PTR = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class LoraDesc(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("n", _I64), ("k", _I64), ("rank", _I32), ("adapters", _I32), ("dtype", _I32),
                ("dtype_y", _I32), ("ldx", _I64), ("ldw", _I64), ("ldy", _I64), ("flags", ctypes.c_uint32), ("tile_n", _I32), ("stages", _I32),
                ("max_ctas", _I32), ("wait_timeout_ns", ctypes.c_uint64)]


class LoraArgs(ctypes.Structure):
    _fields_ = [("x", _PTR), ("w", _PTR), ("a", _PTR), ("lda", _I64), ("stride_a", _I64), ("b", _PTR), ("ldb", _I64),
                ("stride_b", _I64), ("adapter", _PTR), ("scale", _PTR), ("y", _PTR)]


class LoraPlanInfo(ctypes.Structure):
    _fields_ = [("product", GemmPlanInfo), ("steps_per_adapter", _I32), ("max_adapters_per_tile", _I32),
                ("shrink_k_split", _I32), ("shrink_grid", _I32), ("product_k_split", _I32), ("reserved0", _I32),
                ("workspace_bytes", _I64)]


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = [("tokens", _I32), ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("rot_dim", _I32),
                ("interleaved", _I32), ("norm", _I32), ("dtype", _I32), ("eps", _F32), ("table_rows", _I32),
                ("table", _PTR), ("positions", _PTR), ("q_weight", _PTR), ("k_weight", _PTR), ("q", _PTR), ("k", _PTR),
                ("q_token", _I64), ("q_head", _I64), ("k_token", _I64), ("k_head", _I64),
                ("q_out", _PTR), ("k_out", _PTR),
                ("q_out_token", _I64), ("q_out_head", _I64), ("k_out_token", _I64), ("k_out_head", _I64),
                ("v", _PTR), ("v_token", _I64), ("v_head", _I64), ("k_cache", _PTR), ("v_cache", _PTR),
                ("k_page", _I64), ("k_place", _I64), ("k_chead", _I64), ("v_page", _I64), ("v_place", _I64), ("v_chead", _I64),
                ("slots", _PTR), ("num_pages", _I64), ("page_size", _I32), ("dtype_cache", _I32),
                ("k_scale", _F32), ("v_scale", _F32)]


class QkNormRopeGrads(ctypes.Structure):
    _fields_ = [("dq_out", _PTR), ("dk_out", _PTR),
                ("dq_out_token", _I64), ("dq_out_head", _I64), ("dk_out_token", _I64), ("dk_out_head", _I64),
                ("dq", _PTR), ("dk", _PTR), ("dq_token", _I64), ("dq_head", _I64), ("dk_token", _I64), ("dk_head", _I64),
                ("dq_weight", _PTR), ("dk_weight", _PTR), ("workspace", _PTR), ("workspace_bytes", _I64)]


class PagedAttnDesc(ctypes.Structure):
    _fields_ = [("max_batch", _I32), ("heads", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("page_size", _I32),
                ("dtype", _I32), ("dtype_cache", _I32), ("window", _I32), ("max_ctas", _I32)]


class PagedAttnPlanInfo(ctypes.Structure):
    _fields_ = [("grid", _I32), ("tile_tokens", _I32), ("head_groups", _I32), ("smem_bytes", _I32),
                ("workspace_bytes", _I64)]


class PagedAttnArgs(ctypes.Structure):
    _fields_ = [("batch", _I32), ("table_width", _I32), ("q", _PTR), ("q_batch", _I64), ("q_head", _I64),
                ("k_cache", _PTR), ("v_cache", _PTR), ("k_page", _I64), ("k_place", _I64), ("k_head", _I64),
                ("v_page", _I64), ("v_place", _I64), ("v_head", _I64), ("num_pages", _I64),
                ("block_table", _PTR), ("table_stride", _I64), ("lengths", _PTR),
                ("out", _PTR), ("out_batch", _I64), ("out_head", _I64), ("lse", _PTR),
                ("scale", _F32), ("k_scale", _F32), ("v_scale", _F32)]


def serving_header_functions():
    """Names of the functions include/serving.h declares."""
    text = open(SERVING_HEADER).read()
    return sorted(set(re.findall(r"^(?:gemm_status_t|int64_t)\s+(\w+)\s*\(", text, re.M)))


_declared = None


def _lib():
    """The library with the serving functions' signatures declared."""
    global _declared
    if _declared is None:
        L = lib()
        ref = ctypes.POINTER
        for name, args in (("lora_plan_create", [ref(_PTR), ref(LoraDesc)]), ("lora_plan_info", [_PTR, ref(LoraPlanInfo)]),
                           ("lora_run", [_PTR, ref(LoraArgs), _PTR]), ("lora_sync_status", [_PTR, _PTR, ref(GemmDeviceError)]),
                           ("lora_plan_destroy", [_PTR]), ("qk_norm_rope_run", [ref(QkNormRopeArgs), _PTR]),
                           ("qk_norm_rope_backward", [ref(QkNormRopeArgs), ref(QkNormRopeGrads), _PTR]),
                           ("paged_attn_plan_create", [ref(_PTR), ref(PagedAttnDesc)]),
                           ("paged_attn_plan_info", [_PTR, ref(PagedAttnPlanInfo)]),
                           ("paged_attn_run", [_PTR, ref(PagedAttnArgs), _PTR]), ("paged_attn_plan_destroy", [_PTR])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        _use_native_facts()
        _use_device_query()
        L.qk_norm_rope_backward_workspace.argtypes, L.qk_norm_rope_backward_workspace.restype = [], _I64
        _declared = L
    return _declared


def _check(status, where):
    if status != GEMM_OK:
        raise GemmError(status, where)


def _no_device():
    return -1


_current_device = _no_device      # the device that work goes to (a stream handle does not tell); -1: there is none


def _use_device_query():
    global _current_device
    import torch
    if torch.cuda.is_available():
        _current_device = torch._C._cuda_getDevice


def _python_facts(*tensors):
    """What a call's checks depend on: everything about its tensors but their addresses and contents."""
    return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.get_device()) for t in tensors])


def _python_fill(args, offsets, *tensors):
    """Writes each tensor's data address (None: 0) at its byte offset of a ctypes structure."""
    for off, t in zip(offsets, tensors):
        _PTR.from_buffer(args, off).value = None if t is None else t.data_ptr()


_facts, _fill = _python_facts, _python_fill


def _use_native_facts():
    """Takes the two functions above from the compiled extension, when it was built for this torch."""
    global _facts, _fill
    import torch
    try:
        from . import _tensor_facts as native
    except ImportError:
        return
    if native.torch_version == torch.__version__.split("+")[0]:
        _facts, _fill = native.facts, native.fill


def _keep(table, key, value):
    """table[key] = value; a table of checked layouts stays small however many there are."""
    if len(table) >= 1024:
        table.clear()
    table[key] = value
    return value


def _as_current(stream, device):
    """Makes the stream of a handle torch's current one: what torch allocates meanwhile is that stream's, to be used again
    only in its order, and in a capture of that stream the graph's."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device))


def _offsets(cls, *names):
    return tuple([getattr(cls, n).offset for n in names])


def _need(cond, text):
    if not cond:
        raise ValueError(text)


def _rows_ok(t, name):
    _need(t.shape[-1] <= 1 or t.stride(-1) == 1, "%s: the last dimension must be contiguous" % name)


def _steps(t, *dims):
    """Strides of a tensor's dimensions; that of one element is never used and may be anything, so it counts as 0."""
    return [t.stride(d) if t.shape[d] > 1 else 0 for d in dims]


def _apart(t, dim, name):
    """A stride that the library takes 0 of for "packed": a tensor that repeats one row or matrix is refused."""
    _need(t.shape[dim] <= 1 or t.stride(dim) != 0, "%s: dimension %d is expanded (stride 0); a copy is needed" % (name, dim))
    return _steps(t, dim)[0]


class _Plan:
    """A created plan (owns the C handle) of the device that was current; use as a context manager or call close()."""

    _destroy = None
    handle = None
    device = -1

    def close(self):
        if self.handle is not None:
            getattr(_lib(), self._destroy)(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- low-rank adapters beside a projection

def _torch_types():
    import torch
    return {GEMM_BF16: torch.bfloat16, GEMM_F16: torch.float16, GEMM_F32: torch.float32, GEMM_E4M3: torch.float8_e4m3fn}


class LoraPlan(_Plan):
    """Y = X W^T + scale_i (X A_i^T) B_i^T with i = adapter[token]; a negative i: the projection alone.

    X [tokens, k], W [n, k], A [adapters, rank, k], B [adapters, n, rank], Y [tokens, n]; X, W, A and B of one 16-bit type;
    every run has exactly `tokens` tokens, on the device that was current when the plan was made.  Rows may be padded (ldx,
    ldw, ldy in elements, 0 = packed; A's and B's strides are taken from the tensors, which must not be expanded).
    """

    _destroy = "lora_plan_destroy"
    captured = False      # lora_matmul: used while its stream was captured,
    last_use = 0          # and when

    def __init__(self, tokens, n, k, *, rank, adapters, dtype=GEMM_BF16, dtype_y=None, ldx=0, ldw=0, ldy=0, flags=0,
                 tile_n=0, stages=0, max_ctas=0, wait_timeout_ns=0):
        d = LoraDesc()
        d.tokens, d.n, d.k, d.rank, d.adapters = tokens, n, k, rank, adapters
        d.dtype, d.dtype_y = dtype, dtype if dtype_y is None else dtype_y
        d.ldx, d.ldw, d.ldy = ldx, ldw, ldy
        d.flags, d.tile_n, d.stages, d.max_ctas, d.wait_timeout_ns = flags, tile_n, stages, max_ctas, wait_timeout_ns
        h = _PTR()
        _check(_lib().lora_plan_create(ctypes.byref(h), ctypes.byref(d)), "lora_plan_create")
        self.handle, self.desc, self.device = h, d, _current_device()
        self.info = LoraPlanInfo()
        _check(_lib().lora_plan_info(h, ctypes.byref(self.info)), "lora_plan_info")
        self._args = {}

    def _checked(self, x, w, a, b, adapter, y, scale):
        import torch
        d = self.desc
        types = _torch_types()
        for name, t, shape, kind in (("x", x, (d.tokens, d.k), types[d.dtype]), ("w", w, (d.n, d.k), types[d.dtype]),
                                     ("a", a, (d.adapters, d.rank, d.k), types[d.dtype]),
                                     ("b", b, (d.adapters, d.n, d.rank), types[d.dtype]),
                                     ("adapter", adapter, (d.tokens,), torch.int32), ("y", y, (d.tokens, d.n), types[d.dtype_y]),
                                     ("scale", scale, (d.adapters,), torch.float32)):
            if t is None:
                continue
            if t.dtype != kind:
                raise TypeError("%s: %s expected, got %s" % (name, kind, t.dtype))
            _need(tuple(t.shape) == shape, "%s: shape %s expected, got %s" % (name, shape, tuple(t.shape)))
            _need(t.is_cuda and t.get_device() == self.device, "%s: must be on the plan's CUDA device, %d" % (name, self.device))
            _rows_ok(t, name)
        for name, t, ld, cols in (("x", x, d.ldx, d.k), ("w", w, d.ldw, d.k), ("y", y, d.ldy, d.n)):
            _need(t.shape[0] <= 1 or t.stride(0) == (ld or cols), "%s: rows %d apart, the plan has %d" % (name, t.stride(0), ld or cols))
        g = LoraArgs()
        g.lda, g.stride_a, g.ldb, g.stride_b = _apart(a, 1, "a"), _apart(a, 0, "a"), _apart(b, 1, "b"), _apart(b, 0, "b")
        return g

    def run(self, x, w, a, b, adapter, y, scale=None, stream=None):
        """Enqueue on `stream` (default: torch's current stream)."""
        return self._run(_facts(x, w, a, b, adapter, y, scale), x, w, a, b, adapter, y, scale, current_stream_handle() if stream is None else stream)

    def _run(self, key, x, w, a, b, adapter, y, scale, stream):
        checked = self._args.get(key)
        if checked is None:
            checked = _keep(self._args, key, self._checked(x, w, a, b, adapter, y, scale))
        g = LoraArgs.from_buffer_copy(checked)
        _fill(g, _LORA_PTRS, x, w, a, b, adapter, scale, y)
        status = _declared.lora_run(self.handle, ctypes.byref(g), stream)
        if status:
            raise GemmError(status, "lora_run")
        return y

    def sync_status(self, stream=None):
        """(status, GemmDeviceError): synchronises the stream and reads the device error record."""
        rec = GemmDeviceError()
        s = _lib().lora_sync_status(self.handle, current_stream_handle() if stream is None else stream, ctypes.byref(rec))
        return s, rec


_LORA_PTRS = _offsets(LoraArgs, "x", "w", "a", "b", "adapter", "scale", "y")

# lora_matmul's plans.  Their workspaces grow with the tokens (67 MB at 8192 tokens, 64 adapters and rank 64), so they are
# bounded: those not used for longest go until the rest takes no more than this.
_LORA_PLAN_BYTES = 1 << 30
_LORA_PLAN_COUNT = 256
_lora_plans = {}
_lora_calls = {}          # the plan of a call's layouts
_lora_uses = itertools.count(1)
_lora_lock = threading.Lock()


def _bound_lora_plans(newest):
    """Gives up plans, but never the newest one nor those that a graph may replay."""
    import torch
    size = sum(p.info.workspace_bytes for p in _lora_plans.values())
    count = len(_lora_plans)
    idle = False
    for key, plan in sorted(_lora_plans.items(), key=lambda item: item[1].last_use):
        if size <= _LORA_PLAN_BYTES and count <= _LORA_PLAN_COUNT:
            return
        if plan.captured or plan is newest:
            continue
        if not idle:
            torch.cuda.synchronize()      # their last launches are done
            idle = True
        del _lora_plans[key]
        size -= plan.info.workspace_bytes
        count -= 1
        plan.close()


def _lora_plan_for(x, w, a, b, out, stream, capturing):
    _need(x.dim() == 2 and w.dim() == 2 and a.dim() == 3 and b.dim() == 3 and out.dim() == 2,
          "x [M, K], w [N, K], a [L, R, K], b [L, N, R], out [M, N] expected")
    _rows_ok(x, "x")
    _rows_ok(w, "w")
    device = x.get_device()
    _need(x.is_cuda and device == _current_device(), "x: must be on the current CUDA device")
    (m, k), n = x.shape, w.shape[0]

    def ld(t):      # a single row's stride is never used: any that is a multiple of 16 bytes
        return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8

    key = (device, stream, x.shape, w.shape, a.shape, x.dtype, out.dtype, ld(x), ld(w), ld(out))
    plan = _lora_plans.get(key)
    if plan is None:
        plan = LoraPlan(m, n, k, rank=a.shape[1], adapters=a.shape[0], dtype=_dtype_code(x.dtype), dtype_y=_dtype_code(out.dtype),
                        ldx=ld(x), ldw=ld(w), ldy=ld(out))
        _lora_plans[key] = plan
        if not capturing:
            _bound_lora_plans(plan)
    return plan


def lora_matmul(x, w, a, b, adapter, *, scale=None, out=None, out_dtype=None):
    """Y = X W^T + scale_i (X A_i^T) B_i^T (see LoraPlan).

    Plans are kept per shape, layout, device and stream, up to 1 GiB of workspaces: the first call of a shape, or of one that
    was given up since, allocates and may wait for the device (a server with few batch sizes makes LoraPlans instead).  Plans
    that a capture used are kept for good; graphs captured on one stream share them, so replay those one after the other (or
    give each a LoraPlan of its own).  Calls may come from several threads.
    """
    import torch
    if _declared is None:
        _lib()
    if out is None:
        _need(x.dim() == 2 and w.dim() == 2, "x [M, K], w [N, K] expected")
        out = torch.empty(x.shape[0], w.shape[0], dtype=out_dtype or x.dtype, device=x.device)
    stream = current_stream_handle()
    capturing = torch._C._cuda_isCurrentStreamCapturing()
    facts = _facts(x, w, a, b, adapter, out, scale)
    key = (_current_device(), stream, facts)
    # A call is two launches that share the plan's workspace: no other thread's come between them.
    with _lora_lock:
        plan = _lora_calls.get(key)
        if plan is None or plan.handle is None:
            plan = _keep(_lora_calls, key, _lora_plan_for(x, w, a, b, out, stream, capturing))
        plan.last_use = next(_lora_uses)
        if capturing:
            plan.captured = True
        return plan._run(facts, x, w, a, b, adapter, out, scale, stream)


# ---------------------------------------------------------------- head norms and rotary positions

def rope_table(positions, rot_dim, *, base=10000.0, factor=1.0, scaling="linear", original_positions=None, beta_fast=32.0,
               beta_slow=1.0, attention_factor=None, device="cuda"):
    """cos and sin of every position below `positions`: [positions, 2, rot_dim / 2] fp32, computed in fp64.

    Pair i turns by position * f_i, f_i = base^(-2i / rot_dim) (Su et al., "RoFormer").  `factor` > 1 stretches the table to
    longer contexts, by the published rules:
      "linear"  positions are divided by the factor (Chen et al., position interpolation);
      "base"    the base becomes base * factor^(rot_dim / (rot_dim - 2)): the fastest pair keeps its frequency, the
                slowest is divided by the factor (known as NTK-aware scaling);
      "blend"   pairs that turn at least beta_fast times within original_positions keep f_i, those that turn at most
                beta_slow times get f_i / factor, and those between are blended linearly over the pair index; cos and
                sin are multiplied by attention_factor (default 0.1 ln(factor) + 1), which scales q . k by its square
                (Peng et al., "YaRN", whose bounds and defaults these are).
    """
    import torch
    _need(rot_dim > 0 and rot_dim % 2 == 0 and positions > 0, "rot_dim must be even and positive, positions positive")
    _need(scaling in ("linear", "base", "blend"), "scaling: 'linear', 'base' or 'blend'")
    _need(factor >= 1.0, "factor must be at least 1")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    if scaling == "base" and factor != 1.0:
        _need(rot_dim > 2, "scaling 'base' needs rot_dim above 2")
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    freq = base ** (-i / rot_dim)
    gain = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "blend" and factor != 1.0:
        _need(original_positions is not None and original_positions > 0, "scaling 'blend' needs original_positions")
        # the pair index at which a pair turns `turns` times within original_positions
        at = lambda turns: rot_dim * math.log(original_positions / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
        keep = 1.0 - ((i / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        gain = 0.1 * math.log(factor) + 1.0 if attention_factor is None else attention_factor
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq.to(device)
    return torch.stack((angle.cos() * gain, angle.sin() * gain), 1).float().contiguous()


def _check_rows(name, t, tokens, dim, kind, device):
    if t is None:
        return
    if t.dtype != kind:
        raise TypeError("%s: %s expected, got %s" % (name, kind, t.dtype))
    _need(t.dim() == 3 and t.shape[0] == tokens and t.shape[2] == dim, "%s: [tokens, heads, head_dim] expected, got %s" % (name, tuple(t.shape)))
    _need(t.get_device() == device, "%s: must be on q's CUDA device" % name)
    _rows_ok(t, name)


def _rope_args(here, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm):
    """The fields forward and backward share, checked; everything but addresses.  here: the current device."""
    import torch
    _need(q.dim() == 3 and q.is_cuda, "q: [tokens, heads, head_dim] on a CUDA device expected")
    tokens, heads, dim = q.shape
    dev = q.get_device()
    _need(dev == here, "q: on CUDA device %d, the current one is %d" % (dev, here))
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q: bfloat16 or float16 expected, got %s" % q.dtype)
    _check_rows("q", q, tokens, dim, q.dtype, dev)
    _check_rows("k", k, tokens, dim, q.dtype, dev)
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None:
            _need(norm, "%s: given without norm" % name)
            if t.dtype != q.dtype:
                raise TypeError("%s: %s expected, got %s" % (name, q.dtype, t.dtype))
            _need(tuple(t.shape) == (dim,) and t.is_contiguous() and t.get_device() == dev, "%s: [head_dim], contiguous, on q's device" % name)
    if positions.dtype != torch.int32:
        raise TypeError("positions: int32 expected, got %s" % positions.dtype)
    _need(tuple(positions.shape) == (tokens,) and positions.is_contiguous() and positions.get_device() == dev, "positions: [tokens], contiguous, on q's device")
    if table.dtype != torch.float32:
        raise TypeError("table: float32 expected, got %s" % table.dtype)
    _need(table.dim() == 3 and table.shape[1] == 2 and table.is_contiguous() and table.get_device() == dev, "table: [positions, 2, rot_dim / 2], contiguous, on q's device")
    g = QkNormRopeArgs()
    g.tokens, g.heads, g.kv_heads, g.head_dim, g.rot_dim = tokens, heads, 0 if k is None else k.shape[1], dim, 2 * table.shape[2]
    g.interleaved, g.norm, g.dtype, g.eps, g.table_rows = int(interleaved), int(norm), _dtype_code(q.dtype), eps, table.shape[0]
    g.q_token, g.q_head = _steps(q, 0, 1)
    if k is not None:
        g.k_token, g.k_head = _steps(k, 0, 1)
    return g


def _check_cache(name, cache, kv_heads, dim, like, device):
    import torch
    if cache.dtype not in (like, torch.float8_e4m3fn):
        raise TypeError("%s: %s or float8_e4m3fn expected, got %s" % (name, like, cache.dtype))
    _need(cache.dim() == 4 and cache.shape[2] == kv_heads and cache.shape[3] == dim,
          "%s: [pages, page_size, kv_heads, head_dim] expected, got %s" % (name, tuple(cache.shape)))
    _need(cache.get_device() == device, "%s: must be on q's CUDA device" % name)
    _rows_ok(cache, name)


def _checked_rope(here, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm, q_out, k_out, v, k_cache, v_cache, slots):
    import torch
    g = _rope_args(here, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm)
    dev = q.get_device()
    _check_rows("q_out", q_out, g.tokens, g.head_dim, q.dtype, dev)
    _need(q_out.shape == q.shape, "q_out: q's shape expected")
    g.q_out_token, g.q_out_head = _steps(q_out, 0, 1)
    if k_out is not None:
        _need(k is not None and k_out.shape == k.shape, "k_out: k's shape expected")
        _check_rows("k_out", k_out, g.tokens, g.head_dim, q.dtype, dev)
        g.k_out_token, g.k_out_head = _steps(k_out, 0, 1)
    if k_cache is not None:
        _need(k is not None and v is not None and v_cache is not None and slots is not None, "a cache append needs k, v, k_cache, v_cache and slots")
        _check_rows("v", v, g.tokens, g.head_dim, q.dtype, dev)
        _need(v.shape == k.shape, "v: k's shape expected")
        _check_cache("k_cache", k_cache, g.kv_heads, g.head_dim, q.dtype, dev)
        _check_cache("v_cache", v_cache, g.kv_heads, g.head_dim, q.dtype, dev)
        _need(v_cache.shape == k_cache.shape and v_cache.dtype == k_cache.dtype, "v_cache: k_cache's shape and type expected")
        if slots.dtype != torch.int32:
            raise TypeError("slots: int32 expected, got %s" % slots.dtype)
        _need(tuple(slots.shape) == (g.tokens,) and slots.is_contiguous() and slots.get_device() == dev, "slots: [tokens], contiguous, on q's device")
        g.v_token, g.v_head = _steps(v, 0, 1)
        g.k_page, g.k_place, g.k_chead = _steps(k_cache, 0, 1, 2)
        g.v_page, g.v_place, g.v_chead = _steps(v_cache, 0, 1, 2)
        g.num_pages, g.page_size, g.dtype_cache = k_cache.shape[0], k_cache.shape[1], _dtype_code(k_cache.dtype)
    else:
        _need(v is None and v_cache is None and slots is None, "v, v_cache and slots go with k_cache")
        _need(k is None or k_out is not None, "k needs k_out or a cache")
    return g


_ROPE_PTRS = _offsets(QkNormRopeArgs, "q", "k", "positions", "table", "q_weight", "k_weight", "q_out", "k_out", "v", "k_cache", "v_cache",
                      "slots")
_GRAD_PTRS = _offsets(QkNormRopeGrads, "dq_out", "dk_out", "dq", "dk")
_rope_checked = {}
_rope_backward_checked = {}


def qk_norm_rope(q, k, positions, table, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, norm=True, q_out=None,
                 k_out=None, v=None, k_cache=None, v_cache=None, slots=None, k_scale=1.0, v_scale=1.0, stream=None):
    """RMS norm of every head row of q [tokens, heads, head_dim] and k [tokens, kv_heads, head_dim] (or None), then its
    rotary position, in one pass; returns (q_out, k_out).

    table: from rope_table, its width sets how much of the head is rotated; positions: int32 [tokens].  interleaved:
    pairs of neighbours instead of halves.  norm=False leaves the rows as they are before the rotation; a weight of None
    counts as ones.  q_out and k_out default to new tensors (k_out only without a cache) and may be q and k themselves.
    With k_cache, v_cache [pages, page_size, kv_heads, head_dim] the keys and v's values also go to slots [tokens] (int32:
    page * page_size + place, negative: nowhere); a float8_e4m3fn cache holds them divided by k_scale / v_scale.
    """
    if stream is not None and (q_out is None or k_out is None and k_cache is None) and q.is_cuda and stream != current_stream_handle():
        with _as_current(stream, q.device):
            return qk_norm_rope(q, k, positions, table, q_weight=q_weight, k_weight=k_weight, eps=eps, interleaved=interleaved, norm=norm,
                                q_out=q_out, k_out=k_out, v=v, k_cache=k_cache, v_cache=v_cache, slots=slots, k_scale=k_scale,
                                v_scale=v_scale)
    if q_out is None:
        q_out = q.new_empty(q.shape)
    if k_out is None and k_cache is None and k is not None:
        k_out = k.new_empty(k.shape)
    L = _declared or _lib()
    here = _current_device()
    key = (here, eps, interleaved, norm, _facts(q, k, positions, table, q_weight, k_weight, q_out, k_out, v, k_cache, v_cache, slots))
    checked = _rope_checked.get(key)
    if checked is None:
        checked = _keep(_rope_checked, key, _checked_rope(here, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm, q_out,
                                                          k_out, v, k_cache, v_cache, slots))
    g = QkNormRopeArgs.from_buffer_copy(checked)
    _fill(g, _ROPE_PTRS, q, k, positions, table, q_weight, k_weight, q_out, k_out, v, k_cache, v_cache, slots)
    if k_cache is not None:
        g.k_scale, g.v_scale = k_scale, v_scale
    status = L.qk_norm_rope_run(ctypes.byref(g), current_stream_handle() if stream is None else stream)
    if status:
        raise GemmError(status, "qk_norm_rope")
    return q_out, k_out


def _checked_rope_backward(here, dq_out, dk_out, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm, dq, dk):
    g = _rope_args(here, q, k, positions, table, q_weight, k_weight, eps, interleaved, norm)
    d = QkNormRopeGrads()
    _need((dk_out is None) == (k is None), "dk goes with k")
    for name, t, like in (("dq", dq_out, q), ("dk", dk_out, k), ("dq_out", dq, q), ("dk_out", dk, k)):
        if like is not None:
            _check_rows(name, t, g.tokens, g.head_dim, q.dtype, q.get_device())
            _need(t.shape == like.shape, "%s: the forward input's shape expected" % name)
    d.dq_out_token, d.dq_out_head, d.dq_token, d.dq_head = _steps(dq_out, 0, 1) + _steps(dq, 0, 1)
    if k is not None:
        d.dk_out_token, d.dk_out_head, d.dk_token, d.dk_head = _steps(dk_out, 0, 1) + _steps(dk, 0, 1)
    return g, d


def qk_norm_rope_backward(dq, dk, q, k, positions, table, *, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, norm=True,
                          dq_out=None, dk_out=None, stream=None):
    """Gradients of qk_norm_rope: (of q, of k, of q_weight, of k_weight), the last two fp32 or None without a weight.

    dq, dk: the gradients of the forward's outputs; q, k: the forward's inputs.  dq_out, dk_out: where the gradients of q
    and k go (default: new tensors; may be dq and dk themselves).
    """
    import torch
    if stream is not None and q.is_cuda and stream != current_stream_handle():
        with _as_current(stream, q.device):
            return qk_norm_rope_backward(dq, dk, q, k, positions, table, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                         interleaved=interleaved, norm=norm, dq_out=dq_out, dk_out=dk_out)
    if dq_out is None:
        dq_out = q.new_empty(q.shape)
    if dk_out is None and k is not None:
        dk_out = k.new_empty(k.shape)
    L = _declared or _lib()
    here = _current_device()
    key = (here, eps, interleaved, norm, _facts(dq, dk, q, k, positions, table, q_weight, k_weight, dq_out, dk_out))
    checked = _rope_backward_checked.get(key)
    if checked is None:
        checked = _keep(_rope_backward_checked, key, _checked_rope_backward(here, dq, dk, q, k, positions, table, q_weight, k_weight, eps,
                                                                            interleaved, norm, dq_out, dk_out))
    g, d = QkNormRopeArgs.from_buffer_copy(checked[0]), QkNormRopeGrads.from_buffer_copy(checked[1])
    _fill(g, _ROPE_PTRS[:6], q, k, positions, table, q_weight, k_weight)
    _fill(d, _GRAD_PTRS, dq, dk, dq_out, dk_out)
    dqw = dkw = None
    if norm and (q_weight is not None or k_weight is not None):
        n, device = q.shape[2], q.device
        if q_weight is not None:
            dqw = torch.empty(n, dtype=torch.float32, device=device)
            d.dq_weight = dqw.data_ptr()
        if k_weight is not None and k is not None:
            dkw = torch.empty(n, dtype=torch.float32, device=device)
            d.dk_weight = dkw.data_ptr()
        # of this call alone, so that calls of several threads and graphs do not meet in it
        work = torch.empty(L.qk_norm_rope_backward_workspace(), dtype=torch.uint8, device=device)
        d.workspace, d.workspace_bytes = work.data_ptr(), work.numel()
    _check(L.qk_norm_rope_backward(ctypes.byref(g), ctypes.byref(d), current_stream_handle() if stream is None else stream),
           "qk_norm_rope_backward")
    return dq_out, dk_out, dqw, dkw


# ---------------------------------------------------------------- attention of one token over a paged cache

_ATTN_PTRS = _offsets(PagedAttnArgs, "q", "k_cache", "v_cache", "block_table", "lengths", "out", "lse")


class PagedAttentionPlan(_Plan):
    """softmax(scale q K^T) V of one new token per sequence over a paged cache.

    Holds the workspace of up to `max_batch` sequences; query head h reads kv head h // (heads // kv_heads).  window > 0:
    each token sees the last `window` positions only.  dtype_cache: dtype, or GEMM_E4M3 (values times k_scale / v_scale).
    """

    _destroy = "paged_attn_plan_destroy"

    def __init__(self, max_batch, *, heads, kv_heads, head_dim, page_size, dtype=GEMM_BF16, dtype_cache=None, window=0, max_ctas=0):
        d = PagedAttnDesc()
        d.max_batch, d.heads, d.kv_heads, d.head_dim, d.page_size = max_batch, heads, kv_heads, head_dim, page_size
        d.dtype, d.dtype_cache, d.window, d.max_ctas = dtype, dtype if dtype_cache is None else dtype_cache, window, max_ctas
        h = _PTR()
        _check(_lib().paged_attn_plan_create(ctypes.byref(h), ctypes.byref(d)), "paged_attn_plan_create")
        self.handle, self.desc, self.device = h, d, _current_device()
        self.info = PagedAttnPlanInfo()
        _check(_lib().paged_attn_plan_info(h, ctypes.byref(self.info)), "paged_attn_plan_info")
        self._args = {}

    def _checked(self, q, k_cache, v_cache, block_table, lengths, out, lse):
        import torch
        d = self.desc
        types = _torch_types()
        _need(q.dim() == 3 and q.is_cuda, "q: [batch, heads, head_dim] on a CUDA device expected")
        batch, dev = q.shape[0], q.get_device()
        _need(dev == self.device, "q: must be on the plan's CUDA device, %d" % self.device)
        _need(batch <= d.max_batch, "q: %d sequences, the plan holds %d" % (batch, d.max_batch))
        for name, t in (("q", q), ("out", out)):
            if t.dtype != types[d.dtype]:
                raise TypeError("%s: %s expected, got %s" % (name, types[d.dtype], t.dtype))
            _need(tuple(t.shape) == (batch, d.heads, d.head_dim) and t.get_device() == dev, "%s: [batch, heads, head_dim] of the plan, on q's device" % name)
            _rows_ok(t, name)
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.dtype != types[d.dtype_cache]:
                raise TypeError("%s: %s expected, got %s" % (name, types[d.dtype_cache], t.dtype))
            _check_cache(name, t, d.kv_heads, d.head_dim, types[d.dtype], dev)
            _need(t.shape[1] == d.page_size and t.shape[0] == k_cache.shape[0], "%s: the plan's page size, as many pages as k_cache" % name)
        for name, t, dims in (("block_table", block_table, 2), ("lengths", lengths, 1)):
            if t.dtype != torch.int32:
                raise TypeError("%s: int32 expected, got %s" % (name, t.dtype))
            _need(t.dim() == dims and t.shape[0] == batch and t.get_device() == dev, "%s: one row per sequence, on q's device" % name)
            _rows_ok(t, name)
        if lse is not None:
            if lse.dtype != torch.float32:
                raise TypeError("lse: float32 expected, got %s" % lse.dtype)
            _need(tuple(lse.shape) == (batch, d.heads) and lse.is_contiguous() and lse.get_device() == dev, "lse: [batch, heads], contiguous, on q's device")
        g = PagedAttnArgs()
        g.batch, g.table_width, g.table_stride = batch, block_table.shape[1], _steps(block_table, 0)[0]
        g.q_batch, g.q_head, g.out_batch, g.out_head = _steps(q, 0, 1) + _steps(out, 0, 1)
        g.k_page, g.k_place, g.k_head = _steps(k_cache, 0, 1, 2)
        g.v_page, g.v_place, g.v_head = _steps(v_cache, 0, 1, 2)
        g.num_pages = k_cache.shape[0]
        return g

    def run(self, q, k_cache, v_cache, block_table, lengths, out, *, lse=None, scale=None, k_scale=1.0, v_scale=1.0, stream=None):
        """Enqueue on `stream` (default: torch's current stream); returns out.

        q, out [batch, heads, head_dim]; k_cache, v_cache [pages, page_size, kv_heads, head_dim], any strides with a
        contiguous last dimension; block_table int32 [batch, width]: the pages of each sequence in order; lengths int32
        [batch]; lse: fp32 [batch, heads] for the logarithm of the softmax sums; scale: default head_dim^-0.5.
        """
        key = _facts(q, k_cache, v_cache, block_table, lengths, out, lse)
        checked = self._args.get(key)
        if checked is None:
            checked = _keep(self._args, key, self._checked(q, k_cache, v_cache, block_table, lengths, out, lse))
        g = PagedAttnArgs.from_buffer_copy(checked)
        _fill(g, _ATTN_PTRS, q, k_cache, v_cache, block_table, lengths, out, lse)
        g.scale = self.desc.head_dim ** -0.5 if scale is None else scale
        g.k_scale, g.v_scale = k_scale, v_scale
        status = _declared.paged_attn_run(self.handle, ctypes.byref(g), current_stream_handle() if stream is None else stream)
        if status:
            raise GemmError(status, "paged_attn_run")
        return out
