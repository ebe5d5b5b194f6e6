"""Operators of a feed-forward block (include/feedforward.h).

* :func:`add_rms_norm`, :func:`add_rms_norm_backward`: the residual's addition and its RMS norm in one pass, in 16 bits or as
  E4M3 codes with the scales that the block-scaled products read.
* :class:`GatedPlan`: act(X Wg^T) * (X Wu^T) in one kernel, and its backward pass.
* :func:`int4_matmul`: products of up to 16 tokens with 4-bit weights and group scales, alone or as a gated pair;
  :func:`int4_quantize` makes such weights.

As in the rest of the package this is argument marshalling: shapes, types, strides and devices are checked here, the work is
enqueued by the CUDA library on torch's current stream (or the one given), and errors raise GemmError (from the library) or
ValueError / TypeError (from these checks).  Outputs that are not given, and scratch memory, are allocated by torch for the
stream that the work goes to.  None of these calls enters torch's autograd graph: training calls the backward passes itself,
from an autograd function of its own for instance.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import (GEMM_BF16, GEMM_SCALE_BLOCK_1x128_128x128, GEMM_SCALE_MX_E8M0_32, GEMM_SCALE_NONE, GemmDeviceError,
               GemmError, GemmPlanInfo, _dtype_code, current_stream_handle, serving)
from .serving import _F32, _I32, _I64, _PTR, _as_current, _check, _keep, _need, _offsets, _Plan, _rows_ok, _steps, _torch_types

FEEDFORWARD_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "feedforward.h")
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_NO_ACTIVATION = 3


class AddRmsNormArgs(ctypes.Structure):
    _fields_ = [("tokens", _I32), ("hidden", _I32), ("dtype", _I32), ("scale_mode", _I32), ("eps", _F32), ("reserved0", _I32),
                ("x", _PTR), ("residual", _PTR), ("weight", _PTR), ("sum", _PTR), ("y", _PTR), ("scales", _PTR),
                ("ldx", _I64), ("ld_residual", _I64), ("ld_sum", _I64), ("ldy", _I64), ("ld_scales", _I64)]


class AddRmsNormGrads(ctypes.Structure):
    _fields_ = [("tokens", _I32), ("hidden", _I32), ("dtype", _I32), ("eps", _F32), ("dy", _PTR), ("h", _PTR), ("weight", _PTR),
                ("d_sum", _PTR), ("dh", _PTR), ("d_weight", _PTR), ("workspace", _PTR), ("workspace_bytes", _I64),
                ("ld_dy", _I64), ("ld_h", _I64), ("ld_d_sum", _I64), ("ld_dh", _I64)]


class GatedDesc(ctypes.Structure):
    _fields_ = [("tokens", _I64), ("features", _I64), ("k", _I64), ("activation", _I32), ("dtype", _I32), ("gradients", _I32),
                ("dtype_dw", _I32), ("ldx", _I64), ("ldw", _I64), ("ldh", _I64), ("ld_gate_up", _I64), ("ld_dx", _I64), ("ld_dw", _I64),
                ("flags", ctypes.c_uint32), ("tile_n", _I32), ("stages", _I32), ("max_ctas", _I32), ("wait_timeout_ns", ctypes.c_uint64)]


class GatedPlanInfo(ctypes.Structure):
    _fields_ = [("product", GemmPlanInfo), ("dx", GemmPlanInfo), ("dw", GemmPlanInfo), ("few_tiles", _I32), ("k_split", _I32),
                ("workspace_bytes", _I64)]


class GatedGrads(ctypes.Structure):
    _fields_ = [("d_h", _PTR), ("x", _PTR), ("w", _PTR), ("gate_up", _PTR), ("d_gate_up", _PTR), ("d_x", _PTR), ("d_w", _PTR)]


class Int4MatmulArgs(ctypes.Structure):
    _fields_ = [("tokens", _I32), ("n", _I32), ("k", _I32), ("group", _I32), ("dtype", _I32), ("activation", _I32),
                ("x", _PTR), ("codes", _PTR), ("scales", _PTR), ("zeros", _PTR), ("y", _PTR),
                ("ldx", _I64), ("ld_codes", _I64), ("ld_scales", _I64), ("ld_zeros", _I64), ("ldy", _I64)]


def feedforward_header_functions():
    """Names of the functions include/feedforward.h declares."""
    text = open(FEEDFORWARD_HEADER).read()
    return sorted(set(re.findall(r"^(?:gemm_status_t|int64_t)\s+(\w+)\s*\(", text, re.M)))


_declared = None


def _lib():
    """The library with the feed-forward functions' signatures declared."""
    global _declared
    if _declared is None:
        L = serving._lib()
        ref = ctypes.POINTER
        for name, args in (("add_rms_norm_run", [ref(AddRmsNormArgs), _PTR]), ("add_rms_norm_backward", [ref(AddRmsNormGrads), _PTR]),
                           ("gated_plan_create", [ref(_PTR), ref(GatedDesc)]), ("gated_plan_info", [_PTR, ref(GatedPlanInfo)]),
                           ("gated_run", [_PTR] * 6), ("gated_backward", [_PTR, ref(GatedGrads), _PTR]),
                           ("gated_sync_status", [_PTR, _PTR, ref(GemmDeviceError)]), ("gated_plan_destroy", [_PTR]),
                           ("int4_matmul_run", [ref(Int4MatmulArgs), _PTR])):
            f = getattr(L, name)
            f.argtypes, f.restype = args, ctypes.c_int
        L.add_rms_norm_backward_workspace.argtypes, L.add_rms_norm_backward_workspace.restype = [_I32], _I64
        _declared = L
    return _declared


def _matrix(name, t, shape, kind, device):
    """A [rows, columns] tensor of this shape, type and device whose rows are contiguous and do not overlap; their distance."""
    if t.dtype != kind:
        raise TypeError("%s: %s expected, got %s" % (name, kind, t.dtype))
    _need(tuple(t.shape) == tuple(shape), "%s: shape %s expected, got %s" % (name, tuple(shape), tuple(t.shape)))
    _need(t.is_cuda and t.get_device() == device, "%s: must be on CUDA device %d" % (name, device))
    _rows_ok(t, name)
    step = _steps(t, 0)[0]
    _need(t.shape[0] <= 1 or step >= t.shape[1], "%s: its rows overlap (stride %d); a copy is needed" % (name, step))
    return step


def _vector(name, t, size, kind, device):
    if t is None:
        return
    if t.dtype != kind:
        raise TypeError("%s: %s expected, got %s" % (name, kind, t.dtype))
    _need(tuple(t.shape) == (size,) and t.is_contiguous() and t.get_device() == device, "%s: [%d], contiguous, on x's device" % (name, size))


def _first(name, t, here):
    """The tensor that a call goes by: [rows, columns] of 16-bit elements on the current device."""
    import torch
    _need(t.dim() == 2 and t.is_cuda, "%s: [tokens, columns] on a CUDA device expected" % name)
    _need(t.get_device() == here, "%s: on CUDA device %d, the current one is %d" % (name, t.get_device(), here))
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("%s: bfloat16 or float16 expected, got %s" % (name, t.dtype))
    return t.shape[0], t.shape[1], t.dtype, t.get_device()


# ---------------------------------------------------------------- residual, RMS norm, output in 8 bits

_NORM_PTRS = _offsets(AddRmsNormArgs, "x", "residual", "weight", "sum", "y", "scales")
_NORM_GRAD_PTRS = _offsets(AddRmsNormGrads, "dy", "h", "weight", "d_sum", "dh")
_norm_checked = {}
_norm_backward_checked = {}


def _checked_norm(here, eps, scale_mode, x, weight, residual, sum_out, out, scales):
    import torch
    tokens, hidden, kind, dev = _first("x", x, here)
    g = AddRmsNormArgs()
    g.tokens, g.hidden, g.dtype, g.scale_mode, g.eps = tokens, hidden, _dtype_code(kind), scale_mode, eps
    g.ldx = _matrix("x", x, (tokens, hidden), kind, dev)
    _vector("weight", weight, hidden, kind, dev)
    if residual is not None:
        g.ld_residual = _matrix("residual", residual, (tokens, hidden), kind, dev)
    if sum_out is not None:
        g.ld_sum = _matrix("sum_out", sum_out, (tokens, hidden), kind, dev)
    g.ldy = _matrix("out", out, (tokens, hidden), kind if scale_mode == GEMM_SCALE_NONE else torch.float8_e4m3fn, dev)
    if scale_mode == GEMM_SCALE_BLOCK_1x128_128x128:
        g.ld_scales = _matrix("scales", scales, (tokens, -(-hidden // 128)), torch.float32, dev)
    elif scale_mode == GEMM_SCALE_MX_E8M0_32:
        _vector("scales", scales, -(-tokens // 128) * -(-hidden // 128) * 512, torch.uint8, dev)
    else:
        _need(scales is None, "scales: given without a scale_mode")
    return g


def add_rms_norm(x, weight=None, *, residual=None, eps=1e-6, out=None, sum_out=None, scale_mode=GEMM_SCALE_NONE, scales=None, stream=None):
    """h = x + residual (rounded to x's type), n = h * rsqrt(mean(h^2) + eps) * weight over the rows of x [tokens, hidden];
    returns (out, scales, sum_out).

    scale_mode GEMM_SCALE_NONE: out holds n in x's type, scales is None.  GEMM_SCALE_BLOCK_1x128_128x128: out holds
    float8_e4m3fn codes and scales fp32 [tokens, ceil(hidden / 128)], the a and scale_a of matmul and Plan.run.
    GEMM_SCALE_MX_E8M0_32: codes and the tiled scale bytes (uint8), the A and sf_a of Plan.run_mx.  Codes' rows are a multiple
    of 16 elements apart, others' of 8.  sum_out receives h (new unless given; without a residual only if given) and may be
    residual or x itself; out may be x or residual where sum_out is not.
    """
    import torch
    L = _declared or _lib()
    # tensors made here belong to the stream that the work goes to
    if stream is not None and x.is_cuda and stream != current_stream_handle() and (
            out is None or (sum_out is None and residual is not None) or (scales is None and scale_mode != GEMM_SCALE_NONE)):
        with _as_current(stream, x.device):
            return add_rms_norm(x, weight, residual=residual, eps=eps, out=out, sum_out=sum_out, scale_mode=scale_mode, scales=scales)
    if sum_out is None and residual is not None:
        sum_out = _new_rows(x, x.dtype, 8)
    if out is None:
        out = _new_rows(x, x.dtype, 8) if scale_mode == GEMM_SCALE_NONE else _new_rows(x, torch.float8_e4m3fn, 16)
    if scales is None:
        if scale_mode == GEMM_SCALE_BLOCK_1x128_128x128:
            scales = x.new_empty(x.shape[0], -(-x.shape[1] // 128), dtype=torch.float32)
        elif scale_mode == GEMM_SCALE_MX_E8M0_32:
            scales = x.new_empty(-(-x.shape[0] // 128) * -(-x.shape[1] // 128) * 512, dtype=torch.uint8)
    here = serving._current_device()
    key = (here, eps, scale_mode, serving._facts(x, weight, residual, sum_out, out, scales))
    checked = _norm_checked.get(key)
    if checked is None:
        checked = _keep(_norm_checked, key, _checked_norm(here, eps, scale_mode, x, weight, residual, sum_out, out, scales))
    g = AddRmsNormArgs.from_buffer_copy(checked)
    serving._fill(g, _NORM_PTRS, x, residual, weight, sum_out, out, scales)
    status = L.add_rms_norm_run(ctypes.byref(g), current_stream_handle() if stream is None else stream)
    if status:
        raise GemmError(status, "add_rms_norm")
    return out, scales, sum_out


def _new_rows(like, dtype, to):
    """An empty tensor of like's shape whose rows are a multiple of `to` elements apart."""
    _need(like.dim() == 2, "x: [tokens, columns] expected")
    rows, cols = like.shape
    return _new_matrix(like, rows, cols, -(-cols // to) * to, dtype)


def _new_matrix(like, rows, cols, ld, dtype):
    """An empty [rows, cols] tensor on like's device whose rows are ld elements apart."""
    t = like.new_empty(rows, ld, dtype=dtype)
    return t if ld == cols else t[:, :cols]


def _checked_norm_backward(here, eps, dy, h, weight, d_sum, dh):
    tokens, hidden, kind, dev = _first("h", h, here)
    g = AddRmsNormGrads()
    g.tokens, g.hidden, g.dtype, g.eps = tokens, hidden, _dtype_code(kind), eps
    shape = (tokens, hidden)
    g.ld_h, g.ld_dy, g.ld_dh = _matrix("h", h, shape, kind, dev), _matrix("dy", dy, shape, kind, dev), _matrix("out", dh, shape, kind, dev)
    if d_sum is not None:
        g.ld_d_sum = _matrix("d_sum", d_sum, shape, kind, dev)
    _vector("weight", weight, hidden, kind, dev)
    return g


def add_rms_norm_backward(dy, h, weight=None, *, d_sum=None, eps=1e-6, out=None, stream=None):
    """Gradients of add_rms_norm: (of x and of the residual alike, of weight in fp32 or None without one).

    dy: the gradient of n; h: the forward pass's sum (x itself without a residual); d_sum: the gradient that reaches h along
    the residual.  out: where the gradient goes (default: a new tensor; may be dy, d_sum or h itself).
    """
    import torch
    L = _declared or _lib()
    if stream is not None and h.is_cuda and stream != current_stream_handle():
        with _as_current(stream, h.device):
            return add_rms_norm_backward(dy, h, weight, d_sum=d_sum, eps=eps, out=out)
    if out is None:
        out = _new_rows(h, h.dtype, 8)
    here = serving._current_device()
    key = (here, eps, serving._facts(dy, h, weight, d_sum, out))
    checked = _norm_backward_checked.get(key)
    if checked is None:
        checked = _keep(_norm_backward_checked, key, _checked_norm_backward(here, eps, dy, h, weight, d_sum, out))
    g = AddRmsNormGrads.from_buffer_copy(checked)
    serving._fill(g, _NORM_GRAD_PTRS, dy, h, weight, d_sum, out)
    d_weight = None
    if weight is not None:
        d_weight = torch.empty(h.shape[1], dtype=torch.float32, device=h.device)
        # of this call alone, so that calls of several threads and graphs do not meet in it
        work = torch.empty(L.add_rms_norm_backward_workspace(h.shape[1]), dtype=torch.uint8, device=h.device)
        g.d_weight, g.workspace, g.workspace_bytes = d_weight.data_ptr(), work.data_ptr(), work.numel()
    status = L.add_rms_norm_backward(ctypes.byref(g), current_stream_handle() if stream is None else stream)
    if status:
        raise GemmError(status, "add_rms_norm_backward")
    return out, d_weight


# ---------------------------------------------------------------- a gated pair of projections

class GatedPlan(_Plan):
    """H = act(X Wg^T) * (X Wu^T), W = [Wg; Wu] in one matrix, and its backward pass.

    X [tokens, k], W [2 features, k], H [tokens, features], of one 16-bit type; activation "silu", "gelu" or "gelu_tanh"; every
    run has exactly `tokens` tokens, on the device that was current when the plan was made.  Rows may be padded (ldx, ldw, ldh
    in elements, 0 = packed, multiples of 8).  gradients: the plan also runs backward(); its weights' gradients are of dtype
    or, with dtype_dw=GEMM_F32, fp32.
    """

    _destroy = "gated_plan_destroy"

    def __init__(self, tokens, features, k, *, activation="silu", dtype=GEMM_BF16, gradients=False, dtype_dw=None, ldx=0, ldw=0, ldh=0,
                 ld_gate_up=0, ld_dx=0, ld_dw=0, flags=0, tile_n=0, stages=0, max_ctas=0, wait_timeout_ns=0):
        _need(activation in ACTIVATIONS, "activation: one of %s" % ", ".join(ACTIVATIONS))
        d = GatedDesc()
        d.tokens, d.features, d.k, d.activation, d.dtype = tokens, features, k, ACTIVATIONS[activation], dtype
        d.gradients, d.dtype_dw = int(gradients), dtype if dtype_dw is None else dtype_dw
        padded = -(-k // 8) * 8
        d.ldx, d.ldw, d.ldh, d.ld_gate_up = ldx or k, ldw or k, ldh or features, ld_gate_up or 2 * features
        # gradients that backward() makes itself have rows on 16-byte boundaries
        d.ld_dx, d.ld_dw = ld_dx or padded, ld_dw or padded
        d.flags, d.tile_n, d.stages, d.max_ctas, d.wait_timeout_ns = flags, tile_n, stages, max_ctas, wait_timeout_ns
        h = _PTR()
        _check(_lib().gated_plan_create(ctypes.byref(h), ctypes.byref(d)), "gated_plan_create")
        self.handle, self.desc, self.device = h, d, serving._current_device()
        self.info = GatedPlanInfo()
        _check(_lib().gated_plan_info(h, ctypes.byref(self.info)), "gated_plan_info")
        self._args, self._grads = set(), set()

    def _matrices(self, **tensors):
        d = self.desc
        types = _torch_types()
        shapes = {"x": (d.tokens, d.k, d.ldx), "w": (2 * d.features, d.k, d.ldw), "out": (d.tokens, d.features, d.ldh),
                  "d_out": (d.tokens, d.features, d.ldh), "gate_up": (d.tokens, 2 * d.features, d.ld_gate_up),
                  "d_gate_up": (d.tokens, 2 * d.features, d.ld_gate_up), "dx": (d.tokens, d.k, d.ld_dx), "dw": (2 * d.features, d.k, d.ld_dw)}
        for name, t in tensors.items():
            if t is None:
                continue
            rows, cols, ld = shapes[name]
            step = _matrix(name, t, (rows, cols), types[d.dtype_dw if name == "dw" else d.dtype], self.device)
            _need(rows <= 1 or step == ld, "%s: rows %d apart, the plan has %d" % (name, step, ld))

    def run(self, x, w, out, gate_up=None, stream=None):
        """Enqueue on `stream` (default: torch's current stream); returns out.  gate_up [tokens, 2 features]: receives both
        projections, for backward()."""
        key = serving._facts(x, w, out, gate_up)
        if key not in self._args:
            self._matrices(x=x, w=w, out=out, gate_up=gate_up)
            if len(self._args) >= 1024:
                self._args.clear()
            self._args.add(key)
        status = _declared.gated_run(self.handle, x.data_ptr(), w.data_ptr(), out.data_ptr(), None if gate_up is None else gate_up.data_ptr(),
                                     current_stream_handle() if stream is None else stream)
        if status:
            raise GemmError(status, "gated_run")
        return out

    def backward(self, d_out, x, w, gate_up, dx=None, dw=None, *, d_gate_up=None, need_dx=True, need_dw=True, stream=None):
        """Gradients of run(): (of x, of w), None where it is not needed.  gate_up: what run() kept; d_gate_up: scratch of its
        shape (default: made here), may be gate_up itself, which is then overwritten."""
        if stream is not None and x.is_cuda and stream != current_stream_handle():
            with _as_current(stream, x.device):
                return self.backward(d_out, x, w, gate_up, dx, dw, d_gate_up=d_gate_up, need_dx=need_dx, need_dw=need_dw)
        d = self.desc
        _need(d.gradients == 1, "backward: the plan was made without gradients")
        types = _torch_types()
        if d_gate_up is None:
            d_gate_up = _new_matrix(x, d.tokens, 2 * d.features, d.ld_gate_up, types[d.dtype])
        if dx is None and need_dx:
            dx = _new_matrix(x, d.tokens, d.k, d.ld_dx, types[d.dtype])
        if dw is None and need_dw:
            dw = _new_matrix(x, 2 * d.features, d.k, d.ld_dw, types[d.dtype_dw])
        if not need_dx:
            dx = None
        if not need_dw:
            dw = None
        key = serving._facts(d_out, x, w, gate_up, d_gate_up, dx, dw)
        if key not in self._grads:
            self._matrices(d_out=d_out, x=x, w=w, gate_up=gate_up, d_gate_up=d_gate_up, dx=dx, dw=dw)
            if len(self._grads) >= 1024:
                self._grads.clear()
            self._grads.add(key)
        g = GatedGrads()
        g.d_h, g.x, g.w, g.gate_up, g.d_gate_up = d_out.data_ptr(), x.data_ptr(), w.data_ptr(), gate_up.data_ptr(), d_gate_up.data_ptr()
        g.d_x, g.d_w = None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr()
        _check(_declared.gated_backward(self.handle, ctypes.byref(g), current_stream_handle() if stream is None else stream), "gated_backward")
        return dx, dw

    def sync_status(self, stream=None):
        """(status, GemmDeviceError): synchronises the stream and reads the device error records of the plan's products."""
        rec = GemmDeviceError()
        s = _lib().gated_sync_status(self.handle, current_stream_handle() if stream is None else stream, ctypes.byref(rec))
        return s, rec


# ---------------------------------------------------------------- products of a few tokens with 4-bit weights

_INT4_PTRS = _offsets(Int4MatmulArgs, "x", "codes", "scales", "zeros", "y")
_int4_checked = {}


def _checked_int4(here, group, activation, x, codes, scales, zeros, out):
    import torch
    tokens, k, kind, dev = _first("x", x, here)
    _need(activation is None or activation in ACTIVATIONS, "activation: None or one of %s" % ", ".join(ACTIVATIONS))
    _need(k % 2 == 0, "x: an even number of columns expected (two codes a byte)")
    _need(isinstance(group, int) and group >= 1, "group: a positive number of columns")
    _need(codes.dim() == 2, "codes: [rows, k / 2] expected")
    rows, groups = codes.shape[0], -(-k // group)
    _need(activation is None or rows % 2 == 0, "codes: gates and as many rows more expected")
    g = Int4MatmulArgs()
    g.tokens, g.n, g.k, g.group, g.dtype = tokens, rows if activation is None else rows // 2, k, group, _dtype_code(kind)
    g.activation = _NO_ACTIVATION if activation is None else ACTIVATIONS[activation]
    g.ldx = _matrix("x", x, (tokens, k), kind, dev)
    g.ld_codes = _matrix("codes", codes, (rows, k // 2), torch.uint8, dev)
    g.ld_scales = _matrix("scales", scales, (rows, groups), kind, dev)
    if zeros is not None:
        g.ld_zeros = _matrix("zeros", zeros, (rows, groups), torch.uint8, dev)
    g.ldy = _matrix("out", out, (tokens, g.n), kind, dev)
    return g


def int4_matmul(x, codes, scales, *, group=128, zeros=None, activation=None, out=None, stream=None):
    """p = x W^T with W[j, k] = scales[j, k // group] * (code[j, k] - zeros[j, k // group]) (zeros None: 8); activation: out =
    act(p[:, :n]) * p[:, n:] of a gated pair, W's first half gates.  Returns out.

    x [tokens, k], at most 16 tokens (more go through matmul with weights in another form); codes uint8 [rows, k / 2], rows a
    multiple of 16 bytes apart: column k in the low half of byte k / 2 when k is even, in the high half when it is odd; scales
    [rows, ceil(k / group)] of x's type; zeros uint8, 0..127; group: a multiple of 32.  k up to 94208 with at most 8 tokens, up
    to 45056 with more.
    """
    if out is None:
        _need(x.dim() == 2 and codes.dim() == 2, "x [tokens, k], codes [rows, k / 2] expected")
        if stream is not None and x.is_cuda and stream != current_stream_handle():
            with _as_current(stream, x.device):
                return int4_matmul(x, codes, scales, group=group, zeros=zeros, activation=activation)
        out = x.new_empty(x.shape[0], codes.shape[0] if activation is None else codes.shape[0] // 2)
    L = _declared or _lib()
    here = serving._current_device()
    key = (here, group, activation, serving._facts(x, codes, scales, zeros, out))
    checked = _int4_checked.get(key)
    if checked is None:
        checked = _keep(_int4_checked, key, _checked_int4(here, group, activation, x, codes, scales, zeros, out))
    g = Int4MatmulArgs.from_buffer_copy(checked)
    serving._fill(g, _INT4_PTRS, x, codes, scales, zeros, out)
    status = L.int4_matmul_run(ctypes.byref(g), current_stream_handle() if stream is None else stream)
    if status:
        raise GemmError(status, "int4_matmul")
    return out


def int4_quantize(w, group=128, *, symmetric=True):
    """(codes, scales, zeros) of a 16-bit weight matrix w [rows, k] for int4_matmul, nearest codes: symmetric, code - 8 in -7..7
    and zeros None; otherwise 0..15 between the group's least and largest value (and zero), with a zero point.  k even; codes'
    rows are padded to 16 bytes."""
    import torch
    _need(w.dim() == 2 and w.shape[1] % 2 == 0, "w: [rows, k] with an even k expected")
    rows, k = w.shape
    blocks = torch.nn.functional.pad(w.float(), (0, -k % group)).unflatten(1, (-1, group))
    if symmetric:
        scales = (blocks.abs().amax(2) / 7).to(w.dtype)
        zeros, at = None, 8.0
    else:
        low, high = blocks.amin(2).clamp(max=0), blocks.amax(2).clamp(min=0)
        scales = ((high - low) / 15).to(w.dtype)
        point = torch.where(scales > 0, -low / scales.float(), 0.0).round().clamp(0, 15)
        zeros, at = point.to(torch.uint8), point[:, :, None]
    s = scales.float()[:, :, None]
    q = torch.where(s > 0, blocks / s, 0.0)
    q = (q.round() + at).clamp(1 if symmetric else 0, 15).to(torch.uint8).flatten(1)
    q = torch.nn.functional.pad(q[:, :k], (0, -k % 32))
    return (q[:, 0::2] | (q[:, 1::2] << 4))[:, : k // 2], scales, zeros
