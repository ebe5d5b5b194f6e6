"""Host-side tests of include/feedforward.h (no GPU): the library exports every declared function, the binding's structures have
the header's layout, requests that cannot be served are refused before any device is touched, and int4_quantize is its formula."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg
from dense_gemm_blackwell_gb300 import feedforward as ff

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
AT = 1 << 20        # an aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()


def test_library_exports_every_declared_function():
    names = dg.feedforward_header_functions()
    assert {"add_rms_norm_run", "add_rms_norm_backward", "add_rms_norm_backward_workspace", "gated_plan_create", "gated_plan_info", "gated_run",
            "gated_backward", "gated_sync_status", "gated_plan_destroy", "int4_matmul_run"} == set(names)
    raw = ctypes.CDLL(dg._LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_structures_match_the_header(tmp_path):
    pairs = {"add_rms_norm_args_t": ff.AddRmsNormArgs, "add_rms_norm_grads_t": ff.AddRmsNormGrads, "gated_desc_t": ff.GatedDesc,
             "gated_plan_info_t": ff.GatedPlanInfo, "gated_grads_t": ff.GatedGrads, "int4_matmul_args_t": ff.Int4MatmulArgs}
    lines = []
    for name, cls in pairs.items():
        lines.append('printf("%s - %%zu\\n", sizeof(%s));' % (name, name))
        for field, _ in cls._fields_:
            lines.append('printf("%s %s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field))
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "feedforward.h"\nint main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, value = line.split()
        cls = pairs[name]
        assert int(value) == (ctypes.sizeof(cls) if field == "-" else getattr(cls, field).offset), line


def norm_args(**kw):
    g = ff.AddRmsNormArgs()
    g.tokens, g.hidden, g.dtype, g.scale_mode, g.eps = 4, 64, dg.GEMM_BF16, dg.GEMM_SCALE_NONE, 1e-6
    g.x = g.residual = g.sum = AT
    g.y = AT + 1024
    for name, value in kw.items():
        setattr(g, name, value)
    return g


BLOCK, MX = dg.GEMM_SCALE_BLOCK_1x128_128x128, dg.GEMM_SCALE_MX_E8M0_32


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(hidden=0), dg.GEMM_ERR_INVALID_ARG), (dict(reserved0=1), dg.GEMM_ERR_INVALID_ARG),
    (dict(eps=-1.0), dg.GEMM_ERR_INVALID_ARG), (dict(eps=float("nan")), dg.GEMM_ERR_INVALID_ARG),
    (dict(dtype=dg.GEMM_F32), dg.GEMM_ERR_UNSUPPORTED), (dict(scale_mode=dg.GEMM_SCALE_NV_E4M3_16), dg.GEMM_ERR_UNSUPPORTED),
    (dict(hidden=32769), dg.GEMM_ERR_UNSUPPORTED), (dict(tokens=2 ** 30 + 1), dg.GEMM_ERR_UNSUPPORTED),
    (dict(y=AT + 64, sum=AT + 64), dg.GEMM_ERR_INVALID_ARG), (dict(ldx=63), dg.GEMM_ERR_INVALID_ARG), (dict(x=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(y=0), dg.GEMM_ERR_INVALID_ARG), (dict(scales=AT), dg.GEMM_ERR_INVALID_ARG), (dict(scale_mode=MX), dg.GEMM_ERR_INVALID_ARG),
    (dict(scale_mode=MX, scales=AT, ld_scales=4), dg.GEMM_ERR_INVALID_ARG), (dict(scale_mode=BLOCK, scales=AT, hidden=129, ldx=136, ld_scales=1),
                                                                          dg.GEMM_ERR_INVALID_ARG),
    (dict(x=AT + 8), dg.GEMM_ERR_ALIGNMENT), (dict(ldx=68), dg.GEMM_ERR_ALIGNMENT), (dict(residual=AT + 2), dg.GEMM_ERR_ALIGNMENT),
    (dict(weight=AT + 4), dg.GEMM_ERR_ALIGNMENT), (dict(scale_mode=BLOCK, scales=AT + 2), dg.GEMM_ERR_ALIGNMENT),
    (dict(scale_mode=BLOCK, scales=AT, ldy=72), dg.GEMM_ERR_ALIGNMENT), (dict(scale_mode=MX, scales=AT + 8), dg.GEMM_ERR_ALIGNMENT),
    (dict(hidden=65), dg.GEMM_ERR_ALIGNMENT)])
def test_norm_refuses(change, status):
    assert ff._lib().add_rms_norm_run(ctypes.byref(norm_args(**change)), None) == status


def test_norm_of_nothing():
    assert ff._lib().add_rms_norm_run(ctypes.byref(norm_args(tokens=0, x=0, y=0)), None) == dg.GEMM_OK
    assert ff._lib().add_rms_norm_run(None, None) == dg.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(hidden=0), dg.GEMM_ERR_INVALID_ARG), (dict(dtype=dg.GEMM_E4M3), dg.GEMM_ERR_UNSUPPORTED),
    (dict(hidden=40000), dg.GEMM_ERR_UNSUPPORTED), (dict(tokens=2 ** 30 + 1), dg.GEMM_ERR_UNSUPPORTED), (dict(dy=0), dg.GEMM_ERR_INVALID_ARG), (dict(ld_h=8), dg.GEMM_ERR_INVALID_ARG),
    (dict(d_weight=AT), dg.GEMM_ERR_INVALID_ARG), (dict(d_weight=AT, workspace=AT, workspace_bytes=64), dg.GEMM_ERR_INVALID_ARG),
    (dict(dh=AT + 8), dg.GEMM_ERR_ALIGNMENT), (dict(ld_dy=65), dg.GEMM_ERR_ALIGNMENT), (dict(d_sum=AT, ld_d_sum=66), dg.GEMM_ERR_ALIGNMENT)])
def test_norm_backward_refuses(change, status):
    g = ff.AddRmsNormGrads()
    g.tokens, g.hidden, g.dtype, g.eps = 4, 64, dg.GEMM_F16, 1e-6
    g.dy = g.h = g.dh = AT
    for name, value in change.items():
        setattr(g, name, value)
    assert ff._lib().add_rms_norm_backward(ctypes.byref(g), None) == status


def gated_desc(**kw):
    d = ff.GatedDesc()
    d.tokens, d.features, d.k, d.activation, d.dtype, d.gradients, d.dtype_dw = 32, 64, 128, 0, dg.GEMM_BF16, 1, dg.GEMM_F32
    for name, value in kw.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(features=0), dg.GEMM_ERR_INVALID_ARG), (dict(k=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(activation=3), dg.GEMM_ERR_INVALID_ARG), (dict(gradients=2), dg.GEMM_ERR_INVALID_ARG), (dict(ldx=100), dg.GEMM_ERR_INVALID_ARG),
    (dict(dtype=dg.GEMM_E4M3), dg.GEMM_ERR_UNSUPPORTED), (dict(dtype_dw=dg.GEMM_F16), dg.GEMM_ERR_UNSUPPORTED),
    (dict(features=60), dg.GEMM_ERR_UNSUPPORTED), (dict(flags=dg.GEMM_FLAG_SINGLE_CTA), dg.GEMM_ERR_UNSUPPORTED),
    (dict(tile_n=192), dg.GEMM_ERR_UNSUPPORTED), (dict(k=129), dg.GEMM_ERR_ALIGNMENT), (dict(ldh=68), dg.GEMM_ERR_ALIGNMENT),
    (dict(ld_gate_up=132), dg.GEMM_ERR_ALIGNMENT), (dict(ld_dx=132), dg.GEMM_ERR_ALIGNMENT), (dict(ld_dw=130), dg.GEMM_ERR_ALIGNMENT)])
def test_gated_refuses(change, status):
    h = ctypes.c_void_p()
    assert ff._lib().gated_plan_create(ctypes.byref(h), ctypes.byref(gated_desc(**change))) == status
    assert h.value is None


def test_gated_without_a_plan():
    L = ff._lib()
    assert L.gated_plan_create(None, None) == dg.GEMM_ERR_INVALID_ARG
    assert L.gated_run(None, AT, AT, AT, None, None) == dg.GEMM_ERR_INVALID_ARG
    assert L.gated_backward(None, ctypes.byref(ff.GatedGrads()), None) == dg.GEMM_ERR_INVALID_ARG
    assert L.gated_plan_info(None, ctypes.byref(ff.GatedPlanInfo())) == dg.GEMM_ERR_INVALID_ARG
    assert L.gated_plan_destroy(None) == dg.GEMM_OK
    with pytest.raises(ValueError, match="activation"):
        dg.GatedPlan(4, 64, 64, activation="relu")
    if not torch.cuda.is_available():
        with pytest.raises(dg.GemmError):
            dg.GatedPlan(4, 64, 64)


def int4_args(**kw):
    g = ff.Int4MatmulArgs()
    g.tokens, g.n, g.k, g.group, g.dtype, g.activation = 2, 64, 256, 64, dg.GEMM_BF16, 3
    g.x = g.codes = g.scales = g.y = AT
    for name, value in kw.items():
        setattr(g, name, value)
    return g


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(n=0), dg.GEMM_ERR_INVALID_ARG), (dict(group=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(activation=4), dg.GEMM_ERR_INVALID_ARG), (dict(x=0), dg.GEMM_ERR_INVALID_ARG), (dict(scales=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(ld_scales=3), dg.GEMM_ERR_INVALID_ARG), (dict(ld_codes=127), dg.GEMM_ERR_INVALID_ARG), (dict(ldy=63), dg.GEMM_ERR_INVALID_ARG),
    (dict(tokens=17), dg.GEMM_ERR_UNSUPPORTED), (dict(n=2 ** 30 + 1), dg.GEMM_ERR_UNSUPPORTED), (dict(k=255), dg.GEMM_ERR_UNSUPPORTED), (dict(group=48), dg.GEMM_ERR_UNSUPPORTED),
    (dict(dtype=dg.GEMM_F32), dg.GEMM_ERR_UNSUPPORTED), (dict(codes=AT + 8), dg.GEMM_ERR_ALIGNMENT), (dict(ldx=260), dg.GEMM_ERR_ALIGNMENT),
    (dict(ld_codes=136), dg.GEMM_ERR_ALIGNMENT), (dict(scales=AT + 1), dg.GEMM_ERR_ALIGNMENT), (dict(y=AT + 1), dg.GEMM_ERR_ALIGNMENT)])
def test_int4_refuses(change, status):
    assert ff._lib().int4_matmul_run(ctypes.byref(int4_args(**change)), None) == status


def test_int4_of_nothing():
    assert ff._lib().int4_matmul_run(ctypes.byref(int4_args(tokens=0, x=0)), None) == dg.GEMM_OK
    assert ff._lib().int4_matmul_run(None, None) == dg.GEMM_ERR_INVALID_ARG


def test_the_binding_wants_device_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for call in (lambda: dg.add_rms_norm(x), lambda: dg.add_rms_norm_backward(x, x),
                 lambda: dg.int4_matmul(x, torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("rows,k,group", [(5, 256, 128), (3, 130, 32), (1, 2, 64)])
def test_int4_quantize(symmetric, rows, k, group):
    gen = torch.Generator().manual_seed(rows)
    w = (torch.randn(rows, k, generator=gen) + 0.5).to(torch.bfloat16)
    w[0] = 0
    codes, scales, zeros = dg.int4_quantize(w, group, symmetric=symmetric)
    assert codes.shape == (rows, k // 2) and (rows == 1 or codes.stride(0) % 16 == 0) and scales.shape == (rows, -(-k // group))
    q = torch.stack((codes & 15, codes >> 4), 2).flatten(1).double()
    at = torch.arange(k) // group
    back = (q - (8.0 if zeros is None else zeros.double()[:, at])) * scales.double()[:, at]
    # half a step of the code, the scale's rounding (half a step of bf16) over at most 15 codes, and for the zero point's
    # rounding another half step
    assert ((back - w.double()).abs() <= scales.double()[:, at] * (0.5 + 15 * 2.0 ** -8 + (0.0 if symmetric else 0.5))).all()
    assert (back[0] == 0).all()
