"""Host-side tests of include/serving.h (no GPU): the library exports every declared function, the binding's structures
have the header's layout, requests that cannot be served are refused before any device is touched, and rope_table is
its formulas."""
import ctypes
import math
import os
import shutil
import subprocess
import threading
import time

import numpy as np
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg
from dense_gemm_blackwell_gb300 import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()


def test_library_exports_every_declared_function():
    names = dg.serving_header_functions()
    assert {"lora_plan_create", "lora_run", "lora_sync_status", "lora_plan_destroy", "qk_norm_rope_run", "qk_norm_rope_backward",
            "qk_norm_rope_backward_workspace", "paged_attn_plan_create", "paged_attn_run", "paged_attn_plan_destroy"} <= set(names)
    raw = ctypes.CDLL(dg._LIB_PATH)
    for n in names:
        assert hasattr(raw, n), n


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_structures_match_the_header(tmp_path):
    pairs = {"lora_desc_t": serving.LoraDesc, "lora_args_t": serving.LoraArgs, "lora_plan_info_t": serving.LoraPlanInfo,
             "qk_norm_rope_args_t": serving.QkNormRopeArgs, "qk_norm_rope_grads_t": serving.QkNormRopeGrads,
             "paged_attn_desc_t": serving.PagedAttnDesc, "paged_attn_plan_info_t": serving.PagedAttnPlanInfo,
             "paged_attn_args_t": serving.PagedAttnArgs}
    lines = []
    for name, cls in pairs.items():
        lines.append('printf("%s - %%zu\\n", sizeof(%s));' % (name, name))
        for field, _ in cls._fields_:
            lines.append('printf("%s %s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field))
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "serving.h"\nint main(void) {\n%s\nreturn 0;\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, value = line.split()
        cls = pairs[name]
        assert int(value) == (ctypes.sizeof(cls) if field == "-" else getattr(cls, field).offset), line


def no_device_or_ok(status):
    return status == (dg.GEMM_OK if torch.cuda.is_available() else dg.GEMM_ERR_NO_DEVICE)


def lora_status(**kw):
    d = serving.LoraDesc()
    base = dict(tokens=16, n=64, k=64, rank=16, adapters=4, dtype=dg.GEMM_BF16, dtype_y=dg.GEMM_BF16)
    for name, value in {**base, **kw}.items():
        setattr(d, name, value)
    h = ctypes.c_void_p()
    s = serving._lib().lora_plan_create(ctypes.byref(h), ctypes.byref(d))
    if s == dg.GEMM_OK:
        serving._lib().lora_plan_destroy(h)
    return s


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(n=0), dg.GEMM_ERR_INVALID_ARG), (dict(k=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(rank=0), dg.GEMM_ERR_INVALID_ARG), (dict(adapters=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(rank=12), dg.GEMM_ERR_UNSUPPORTED), (dict(rank=264), dg.GEMM_ERR_UNSUPPORTED),
    (dict(adapters=4097), dg.GEMM_ERR_UNSUPPORTED), (dict(dtype=dg.GEMM_F32), dg.GEMM_ERR_UNSUPPORTED),
    (dict(dtype=dg.GEMM_E4M3), dg.GEMM_ERR_UNSUPPORTED), (dict(dtype_y=dg.GEMM_E4M3), dg.GEMM_ERR_UNSUPPORTED),
    (dict(tokens=65535 * 64 + 1), dg.GEMM_ERR_UNSUPPORTED),
    (dict(flags=dg.GEMM_FLAG_SINGLE_CTA), dg.GEMM_ERR_UNSUPPORTED), (dict(flags=dg.GEMM_FLAG_ACCUM_F16), dg.GEMM_ERR_UNSUPPORTED),
])
def test_lora_plan_refuses(kw, status):
    assert lora_status(**kw) == status


def test_lora_plan_accepts_what_it_documents():
    for kw in (dict(), dict(rank=8), dict(rank=256, adapters=4096), dict(tokens=0), dict(dtype=dg.GEMM_F16, dtype_y=dg.GEMM_F32)):
        assert no_device_or_ok(lora_status(**kw)), kw
    assert serving._lib().lora_plan_create(None, None) == dg.GEMM_ERR_INVALID_ARG
    assert serving._lib().lora_run(None, None, None) == dg.GEMM_ERR_INVALID_ARG
    assert serving._lib().lora_plan_info(None, None) == dg.GEMM_ERR_INVALID_ARG
    assert serving._lib().lora_sync_status(None, None, None) == dg.GEMM_ERR_INVALID_ARG
    assert serving._lib().lora_plan_destroy(None) == dg.GEMM_OK


def rope_args(**kw):
    """A complete forward request on made-up, aligned addresses (never dereferenced: refusals come first)."""
    a = serving.QkNormRopeArgs()
    base = dict(tokens=4, heads=2, kv_heads=1, head_dim=64, rot_dim=64, norm=1, dtype=dg.GEMM_BF16, eps=1e-6, table_rows=8,
                table=1 << 20, positions=1 << 21, q_weight=1 << 22, k_weight=1 << 22, q=1 << 23, k=1 << 24, q_token=192, q_head=64,
                k_token=192, k_head=64, q_out=1 << 25, k_out=1 << 26, q_out_token=128, q_out_head=64, k_out_token=64, k_out_head=64,
                dtype_cache=dg.GEMM_BF16, page_size=16, num_pages=4, k_scale=1.0, v_scale=1.0)
    for name, value in {**base, **kw}.items():
        setattr(a, name, value)
    return a


CACHE = dict(v=1 << 27, v_token=192, v_head=64, k_cache=1 << 28, v_cache=1 << 29, k_page=1024, k_place=64, k_chead=64, v_page=1024,
             v_place=64, v_chead=64, slots=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), dg.GEMM_ERR_INVALID_ARG), (dict(rot_dim=66), dg.GEMM_ERR_INVALID_ARG), (dict(rot_dim=31), dg.GEMM_ERR_INVALID_ARG),
    (dict(head_dim=60, rot_dim=32), dg.GEMM_ERR_UNSUPPORTED), (dict(head_dim=264, rot_dim=64), dg.GEMM_ERR_UNSUPPORTED),
    (dict(dtype=dg.GEMM_F32), dg.GEMM_ERR_UNSUPPORTED), (dict(table=None), dg.GEMM_ERR_INVALID_ARG),
    (dict(positions=None), dg.GEMM_ERR_INVALID_ARG), (dict(table_rows=0), dg.GEMM_ERR_INVALID_ARG), (dict(q=None), dg.GEMM_ERR_INVALID_ARG),
    (dict(q_out=None), dg.GEMM_ERR_INVALID_ARG), (dict(k_out=None), dg.GEMM_ERR_INVALID_ARG), (dict(q=(1 << 23) + 2), dg.GEMM_ERR_ALIGNMENT),
    (dict(q_token=196), dg.GEMM_ERR_ALIGNMENT), (dict(k_out_head=60), dg.GEMM_ERR_ALIGNMENT), (dict(q_weight=(1 << 22) + 8), dg.GEMM_ERR_ALIGNMENT),
    (dict(CACHE, v=None), dg.GEMM_ERR_INVALID_ARG), (dict(CACHE, slots=None), dg.GEMM_ERR_INVALID_ARG),
    (dict(CACHE, v_cache=None), dg.GEMM_ERR_INVALID_ARG), (dict(CACHE, page_size=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(CACHE, dtype_cache=dg.GEMM_F16), dg.GEMM_ERR_UNSUPPORTED), (dict(CACHE, dtype_cache=dg.GEMM_E4M3, k_scale=0.0), dg.GEMM_ERR_INVALID_ARG),
    (dict(CACHE, k_place=68), dg.GEMM_ERR_ALIGNMENT), (dict(CACHE, k_cache=(1 << 28) + 8), dg.GEMM_ERR_ALIGNMENT),
])
def test_rope_refuses(kw, status):
    assert serving._lib().qk_norm_rope_run(ctypes.byref(rope_args(**kw)), None) == status


def test_rope_without_work_is_a_no_op():
    assert serving._lib().qk_norm_rope_run(ctypes.byref(rope_args(tokens=0, q=None, k=None)), None) == dg.GEMM_OK
    assert serving._lib().qk_norm_rope_run(ctypes.byref(rope_args(heads=0, kv_heads=0, q=None, k=None)), None) == dg.GEMM_OK
    assert serving._lib().qk_norm_rope_run(None, None) == dg.GEMM_ERR_INVALID_ARG


@pytest.mark.parametrize("args,grads,status", [
    (dict(q_weight=None), dict(dq_weight=1 << 20), dg.GEMM_ERR_INVALID_ARG),      # a gradient of no weight
    (dict(norm=0), dict(dq_weight=1 << 20), dg.GEMM_ERR_INVALID_ARG),
    (dict(), dict(dq_weight=1 << 20, workspace=None), dg.GEMM_ERR_INVALID_ARG),
    (dict(), dict(dq_weight=1 << 20, workspace_bytes=64), dg.GEMM_ERR_INVALID_ARG),
    (dict(), dict(dq=None), dg.GEMM_ERR_INVALID_ARG), (dict(), dict(dk_out=None), dg.GEMM_ERR_INVALID_ARG),
    (dict(), dict(dq_token=12), dg.GEMM_ERR_ALIGNMENT),
])
def test_rope_backward_refuses(args, grads, status):
    g = serving.QkNormRopeGrads()
    base = dict(dq_out=1 << 23, dk_out=1 << 24, dq=1 << 25, dk=1 << 26, dq_out_token=128, dq_out_head=64, dk_out_token=64, dk_out_head=64,
                dq_token=128, dq_head=64, dk_token=64, dk_head=64, workspace=1 << 27,
                workspace_bytes=serving._lib().qk_norm_rope_backward_workspace())
    for name, value in {**base, **grads}.items():
        setattr(g, name, value)
    assert serving._lib().qk_norm_rope_backward(ctypes.byref(rope_args(**args)), ctypes.byref(g), None) == status


def attn_status(**kw):
    d = serving.PagedAttnDesc()
    base = dict(max_batch=4, heads=8, kv_heads=2, head_dim=64, page_size=16, dtype=dg.GEMM_BF16, dtype_cache=dg.GEMM_BF16)
    for name, value in {**base, **kw}.items():
        setattr(d, name, value)
    h = ctypes.c_void_p()
    s = serving._lib().paged_attn_plan_create(ctypes.byref(h), ctypes.byref(d))
    if s == dg.GEMM_OK:
        serving._lib().paged_attn_plan_destroy(h)
    return s


@pytest.mark.parametrize("kw,status", [
    (dict(max_batch=-1), dg.GEMM_ERR_INVALID_ARG), (dict(heads=7), dg.GEMM_ERR_INVALID_ARG), (dict(kv_heads=0), dg.GEMM_ERR_INVALID_ARG),
    (dict(page_size=0), dg.GEMM_ERR_INVALID_ARG), (dict(window=-1), dg.GEMM_ERR_INVALID_ARG), (dict(head_dim=60), dg.GEMM_ERR_UNSUPPORTED),
    (dict(head_dim=264), dg.GEMM_ERR_UNSUPPORTED), (dict(head_dim=72, dtype_cache=dg.GEMM_E4M3), dg.GEMM_ERR_UNSUPPORTED),
    (dict(dtype=dg.GEMM_F32), dg.GEMM_ERR_UNSUPPORTED), (dict(dtype_cache=dg.GEMM_F16), dg.GEMM_ERR_UNSUPPORTED),
    (dict(dtype_cache=dg.GEMM_E5M2), dg.GEMM_ERR_UNSUPPORTED),
])
def test_paged_attn_plan_refuses(kw, status):
    assert attn_status(**kw) == status


def test_paged_attn_plan_accepts_what_it_documents():
    for kw in (dict(), dict(head_dim=8), dict(head_dim=256, dtype=dg.GEMM_F16, dtype_cache=dg.GEMM_E4M3), dict(page_size=1), dict(max_batch=0)):
        assert no_device_or_ok(attn_status(**kw)), kw
    assert serving._lib().paged_attn_run(None, None, None) == dg.GEMM_ERR_INVALID_ARG
    assert serving._lib().paged_attn_plan_destroy(None) == dg.GEMM_OK


def test_python_layer_refuses_host_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dg.qk_norm_rope(x, None, torch.zeros(4, dtype=torch.int32), torch.zeros(8, 2, 32))


class Layout:
    """What the binding's checks ask of a tensor on CUDA device `device`; nothing is allocated."""

    def __init__(self, shape, dtype, stride=None, device=0):
        self.shape, self.dtype, self.device_index = tuple(shape), dtype, device
        self.strides = tuple(torch.empty(shape, device="meta").stride() if stride is None else stride)
        self.is_cuda = True

    def stride(self, dim=None):
        return self.strides if dim is None else self.strides[dim]

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return self.strides == torch.empty(self.shape, device="meta").stride()


def lora_layouts(tokens=16, n=64, k=128, rank=16, adapters=4, **other):
    """(a plan that owns nothing, the layouts of one run's tensors), with the tensors in `other` in place of the packed ones."""
    plan = object.__new__(dg.LoraPlan)
    plan.desc = serving.LoraDesc(tokens=tokens, n=n, k=k, rank=rank, adapters=adapters, dtype=dg.GEMM_BF16, dtype_y=dg.GEMM_BF16)
    plan.device = 0
    half = torch.bfloat16
    kinds = dict(x=Layout((tokens, k), half), w=Layout((n, k), half), a=Layout((adapters, rank, k), half), b=Layout((adapters, n, rank), half),
                 adapter=Layout((tokens,), torch.int32), y=Layout((tokens, n), half), scale=Layout((adapters,), torch.float32))
    return plan, {**kinds, **other}


def test_lora_refuses_expanded_adapters():
    """A stride of 0 would count as packed in the library, which then reads past the one matrix there is."""
    half = torch.bfloat16
    plan, good = lora_layouts()
    assert plan._checked(**good).stride_a == 16 * 128
    for bad in (dict(a=Layout((4, 16, 128), half, (0, 128, 1))), dict(a=Layout((4, 16, 128), half, (128, 0, 1))),
                dict(b=Layout((4, 64, 16), half, (0, 16, 1))), dict(b=Layout((4, 64, 16), half, (16, 0, 1)))):
        with pytest.raises(ValueError):
            plan._checked(**{**good, **bad})
    plan, one = lora_layouts(adapters=1)            # one adapter: nothing is repeated
    plan._checked(**one)


def attn_layouts(batch=3, heads=8, kv=2, dim=64, page=16, **other):
    """The same for the attention."""
    plan = object.__new__(dg.PagedAttentionPlan)
    plan.desc = serving.PagedAttnDesc(max_batch=batch, heads=heads, kv_heads=kv, head_dim=dim, page_size=page, dtype=dg.GEMM_BF16,
                                      dtype_cache=dg.GEMM_BF16)
    plan.device = 0
    half = torch.bfloat16
    kinds = dict(q=Layout((batch, heads, dim), half), k_cache=Layout((9, page, kv, dim), half), v_cache=Layout((9, page, kv, dim), half),
                 block_table=Layout((batch, 4), torch.int32), lengths=Layout((batch,), torch.int32), out=Layout((batch, heads, dim), half),
                 lse=Layout((batch, heads), torch.float32))
    return plan, {**kinds, **other}


def rope_layouts(tokens=5, heads=8, kv=2, dim=64, **other):
    """The tensors and options of a forward pass's checks."""
    half = torch.bfloat16
    kinds = dict(q=Layout((tokens, heads, dim), half), k=Layout((tokens, kv, dim), half), positions=Layout((tokens,), torch.int32),
                 table=Layout((32, 2, dim // 2), torch.float32), q_weight=None, k_weight=None, eps=1e-6, interleaved=False, norm=True,
                 q_out=Layout((tokens, heads, dim), half), k_out=Layout((tokens, kv, dim), half), v=None, k_cache=None, v_cache=None, slots=None)
    return {**kinds, **other}


def test_plans_refuse_tensors_of_another_device():
    """All tensors of a call on one device, but not on the one that the plan's workspace and the stream belong to."""
    for plan, good in (lora_layouts(), attn_layouts()):
        plan._checked(**good)
        for t in good.values():
            t.device_index = 1
        with pytest.raises(ValueError):
            plan._checked(**good)


def test_head_norms_refuse_tensors_of_another_device_than_the_current_one():
    good = rope_layouts()
    assert serving._checked_rope(0, **good).tokens == 5
    with pytest.raises(ValueError):
        serving._checked_rope(1, **good)
    shared = {n: good[n] for n in ("q", "k", "positions", "table", "q_weight", "k_weight", "eps", "interleaved", "norm")}
    grads = dict(dq_out=good["q"], dk_out=good["k"], dq=good["q_out"], dk=good["k_out"])
    serving._checked_rope_backward(0, **shared, **grads)
    with pytest.raises(ValueError):
        serving._checked_rope_backward(1, **shared, **grads)


def test_the_current_device_is_part_of_what_is_checked(monkeypatch):
    """Checks are kept by layout and current device: the same layouts under another one are checked again."""
    current = [0]

    def check(here, *rest):
        raise KeyError(here)

    good = rope_layouts()
    names = ("q", "k", "positions", "table", "q_weight", "k_weight", "q_out", "k_out", "v", "k_cache", "v_cache", "slots")
    kept = (0, 1e-6, False, True, serving._python_facts(*[good[n] for n in names]))
    serving._lib()
    monkeypatch.setattr(serving, "_facts", serving._python_facts)
    monkeypatch.setattr(serving, "_current_device", lambda: current[0])
    monkeypatch.setattr(serving, "_rope_checked", {kept: "found"})
    monkeypatch.setattr(serving, "_checked_rope", check)
    run = lambda: dg.qk_norm_rope(good["q"], good["k"], good["positions"], good["table"], q_out=good["q_out"], k_out=good["k_out"])  # noqa: E731
    with pytest.raises(TypeError):          # found: text is no structure to copy
        run()
    current[0] = 1
    with pytest.raises(KeyError):           # checked
        run()


def test_strides_of_single_elements_do_not_matter():
    """A dimension of one element may have any stride (tensors from other libraries often say 1): it is never used, and must
    not fail the checks of alignment."""
    half = torch.bfloat16
    plan, args = attn_layouts(batch=1, heads=1, kv=1, page=1, q=Layout((1, 1, 64), half, (1, 1, 1)), out=Layout((1, 1, 64), half, (3, 5, 1)),
                              k_cache=Layout((9, 1, 1, 64), half, (64, 1, 1, 1)), v_cache=Layout((9, 1, 1, 64), half, (64, 7, 7, 1)),
                              block_table=Layout((1, 4), torch.int32, (-1, 1)))
    g = plan._checked(**args)
    names = ("q_batch", "q_head", "out_batch", "out_head", "k_place", "k_head", "v_place", "v_head", "table_stride")
    assert [getattr(g, n) for n in names] == [0] * len(names) and g.k_page == 64
    row = Layout((1, 1, 64), half, (1, 1, 1))
    g = serving._checked_rope(0, **rope_layouts(tokens=1, heads=1, kv=1, q=row, k=row, q_out=row, k_out=row, v=row,
                                                k_cache=Layout((9, 1, 1, 64), half, (64, 1, 1, 1)), v_cache=Layout((9, 1, 1, 64), half, (64, 1, 1, 1)),
                                                slots=Layout((1,), torch.int32)))
    assert not any(getattr(g, n) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "q_out_token", "k_out_head", "k_place", "v_chead"))
    plan, args = lora_layouts(tokens=1, n=1, adapters=1, x=Layout((1, 128), half, (1, 1)), w=Layout((1, 128), half, (1, 1)),
                              a=Layout((1, 16, 128), half, (1, 128, 1)), b=Layout((1, 1, 16), half, (1, 1, 1)), y=Layout((1, 1), half, (1, 1)))
    g = plan._checked(**args)
    assert (g.stride_a, g.lda, g.stride_b, g.ldb) == (0, 128, 0, 0)


class StandInPlan:
    """Counts as a LoraPlan of 300 bytes."""

    made = []
    captured, last_use = False, 0

    def __init__(self, tokens, n, k, **kw):
        self.kw = kw
        self.info = type("Info", (), {"workspace_bytes": 300})
        self.tokens, self.handle = tokens, 1
        StandInPlan.made.append(self)

    def _run(self, facts, x, *rest):
        assert self.handle and self.tokens == x.shape[0]
        return x.shape[0]

    def close(self):
        self.handle = None

    @property
    def open(self):
        return self.handle is not None


@pytest.fixture
def stand_in_plans(monkeypatch):
    """(call lora_matmul for a number of tokens, a list whose last element says whether the stream is captured)"""
    state, waited = [False], []
    monkeypatch.setattr(StandInPlan, "made", [])
    monkeypatch.setattr(serving, "LoraPlan", StandInPlan)
    monkeypatch.setattr(serving, "_current_device", lambda: 0)
    monkeypatch.setattr(serving, "current_stream_handle", lambda: 7)
    monkeypatch.setattr(serving, "_facts", serving._python_facts)
    monkeypatch.setattr(serving, "_lora_plans", {})
    monkeypatch.setattr(serving, "_lora_calls", {})
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state[-1], raising=False)
    serving._lib()
    monkeypatch.setattr(torch.cuda, "synchronize", lambda *a: waited.append([p.open for p in StandInPlan.made]))

    def call(tokens):
        half = torch.bfloat16
        x, w, y = Layout((tokens, 64), half), Layout((32, 64), half), Layout((tokens, 32), half)
        assert dg.lora_matmul(x, w, Layout((2, 8, 64), half), Layout((2, 32, 8), half), Layout((tokens,), torch.int32), out=y) == tokens

    return call, state, waited


def test_lora_matmul_takes_single_rows_of_any_width(stand_in_plans):
    """A row alone has no neighbour to be 16 bytes apart from."""
    half = torch.bfloat16
    x, w, y = Layout((1, 1001), half), Layout((1543, 1001), half, (1008, 1)), Layout((1, 1543), half)
    dg.lora_matmul(x, w, Layout((2, 8, 1001), half, (8064, 1008, 1)), Layout((2, 1543, 8), half), Layout((1,), torch.int32), out=y)
    assert [StandInPlan.made[0].kw[n] for n in ("ldx", "ldw", "ldy")] == [1008, 1008, 1544]


def test_lora_matmul_bounds_its_plans(stand_in_plans, monkeypatch):
    """Ever new token counts: the oldest plans are given up once the device is idle, those that a graph may replay are not."""
    call, state, waited = stand_in_plans
    monkeypatch.setattr(serving, "_LORA_PLAN_BYTES", 1000)
    for tokens in (1, 2, 3, 1, 4):
        call(tokens)
    assert [p.tokens for p in StandInPlan.made if p.open] == [1, 3, 4]           # 2 was used least recently
    assert waited == [[True] * 4]                                                # the wait came before the first was closed
    state.append(True)
    call(3)                                                                      # captured: nothing is freed or waited for
    call(5)
    assert len(waited) == 1 and [p.tokens for p in StandInPlan.made if p.open] == [1, 3, 4, 5]
    state.append(False)
    for tokens in range(6, 12):
        call(tokens)
    still = [p.tokens for p in StandInPlan.made if p.open]
    assert still == [3, 5, 11] and [p.tokens for p in serving._lora_plans.values()] == still
    call(4)                                                                      # given up before: made anew, and 11 goes for it
    assert len(StandInPlan.made) == 12 and [p.tokens for p in StandInPlan.made if p.open] == [3, 5, 4]
    monkeypatch.setattr(serving, "_LORA_PLAN_BYTES", 100)                        # the last one stays even if it alone is too much
    call(12)
    assert [p.tokens for p in StandInPlan.made if p.open] == [3, 5, 12]
    monkeypatch.setattr(serving, "_LORA_PLAN_BYTES", 1 << 30)
    monkeypatch.setattr(serving, "_LORA_PLAN_COUNT", 4)
    for tokens in range(13, 20):
        call(tokens)
    assert [p.tokens for p in StandInPlan.made if p.open] == [3, 5, 18, 19]


def test_lora_matmul_s_launches_of_one_call_stay_together(stand_in_plans, monkeypatch):
    """No other thread runs a plan while one thread does."""
    call, _, _ = stand_in_plans
    inside, worst = [0], [0]

    def run(self, facts, x, *rest):
        inside[0] += 1
        worst[0] = max(worst[0], inside[0])
        time.sleep(0.002)
        inside[0] -= 1
        return x.shape[0]

    monkeypatch.setattr(StandInPlan, "_run", run)
    threads = [threading.Thread(target=lambda: [call(t) for t in (1, 2, 3)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert worst[0] == 1 and len(StandInPlan.made) == 3


def test_native_tensor_facts_agree_with_the_python_ones():
    """Both tell the same layouts apart and write the same addresses."""
    serving._lib()
    native = pytest.importorskip("dense_gemm_blackwell_gb300._tensor_facts")
    a = torch.zeros(4, 6, 8)
    kinds = [a, a.clone(), a[1:], a[:, ::2], a.transpose(0, 1), a.half(), torch.zeros(4, 6, 8, 1), torch.zeros(()), None,
             torch.zeros(24, 8), a.double(), torch.zeros(4, 6, 8, dtype=torch.int32)]
    for x in kinds:
        for y in kinds:
            for rest in ((), (a, None)):
                same = serving._python_facts(x, *rest) == serving._python_facts(y, *rest)
                assert (native.facts(x, *rest) == native.facts(y, *rest)) == same
    assert native.facts(a, None) != native.facts(None, a)
    assert native.facts(a) != native.facts(a.to("meta"))
    offsets = serving._LORA_PTRS
    one, two = serving.LoraArgs(), serving.LoraArgs()
    tensors = (a, a[2:], None, torch.zeros(0), a.half(), None, a[:, 1:])
    native.fill(one, offsets, *tensors)
    serving._python_fill(two, offsets, *tensors)
    assert bytes(one) == bytes(two) and one.w == a[2:].data_ptr() and one.scale is None
    for bad in (lambda: native.facts(3), lambda: native.facts("x", a), lambda: native.facts(a.to_sparse()), lambda: native.fill(one, (0,), 3),
                lambda: native.fill(one, (0, 8), a), lambda: native.fill(one)):
        with pytest.raises(TypeError):
            bad()
    for off in (-1, ctypes.sizeof(one), 1 << 40):
        with pytest.raises(ValueError):
            native.fill(one, (off,), a)


# ---------------------------------------------------------------- rope_table

def plain_table(positions, freq, gain=1.0):
    a = np.outer(np.arange(positions, dtype=np.float64), freq)
    return np.stack((np.cos(a) * gain, np.sin(a) * gain), 1)


def test_rope_table_is_its_formulas():
    """fp32 values of fp64 cosines: half an fp32 unit of values up to the gain, 2^-24 each; torch and numpy round cos and sin
    differently by at most a few fp64 units of angles below 1e5 (1e5 * 2^-53 = 1.1e-11)."""
    rot, n = 48, 999
    i = np.arange(0, rot, 2)
    plain = 500000.0 ** (-i / rot)
    tol = 2.0 ** -24 + 1e-10

    def check(table, want):
        assert table.dtype == torch.float32 and tuple(table.shape) == (n, 2, rot // 2) and table.is_contiguous()
        assert np.max(np.abs(table.double().numpy() - want)) <= tol * max(1.0, np.max(np.abs(want)))

    check(dg.rope_table(n, rot, base=500000.0, device="cpu"), plain_table(n, plain))
    check(dg.rope_table(n, rot, base=500000.0, factor=4.0, device="cpu"), plain_table(n, plain / 4))
    stretched = (500000.0 * 4 ** (rot / (rot - 2))) ** (-i / rot)
    assert stretched[0] == 1.0 and abs(stretched[-1] / plain[-1] - 0.25) < 1e-12      # fastest kept, slowest divided
    check(dg.rope_table(n, rot, base=500000.0, factor=4.0, scaling="base", device="cpu"), plain_table(n, stretched))
    # blend: pairs by the number of turns within the original context
    orig, factor = 8192, 8.0
    blended = dg.rope_table(n, rot, base=500000.0, factor=factor, scaling="blend", original_positions=orig, device="cpu")
    index = lambda turns: rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(500000.0))  # noqa: E731
    low, high = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rot - 1)
    keep = 1 - np.clip((i / 2 - low) / (high - low), 0, 1)
    turns = orig * plain / (2 * math.pi)
    assert np.all(keep[turns > 80] == 1) and np.all(keep[turns < 0.5] == 0)
    gain = 0.1 * math.log(factor) + 1
    check(blended, plain_table(n, plain * keep + plain / factor * (1 - keep), gain))
    check(dg.rope_table(n, rot, base=500000.0, factor=factor, scaling="blend", original_positions=orig, attention_factor=1.0, device="cpu"),
          plain_table(n, plain * keep + plain / factor * (1 - keep)))


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(positions=0), dict(scaling="other"), dict(factor=0.5),
                                dict(factor=2.0, scaling="blend"), dict(rot_dim=2, factor=2.0, scaling="base")])
def test_rope_table_refuses(kw):
    args = dict(positions=8, rot_dim=8, device="cpu")
    args.update(kw)
    with pytest.raises(ValueError):
        dg.rope_table(args.pop("positions"), args.pop("rot_dim"), **args)
