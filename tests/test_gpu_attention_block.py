"""GPU: the example's attention block runs the serving operators together and agrees with its plain form.

Between the operators activations are rounded to bf16 (2^-9 relative each, in norm): qkv, q and k after the rotation, P, o, and
y, where the plain form keeps fp32; errors of a softmax over few tokens enter once more.  Eight roundings in all: 2^-6.
"""
import importlib.util
import os

import pytest

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


@pytest.fixture(scope="module")
def example():
    dg.build()
    spec = importlib.util.spec_from_file_location("attention_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("batch,steps,sizes", [
    (1, 3, dict(hidden=512, heads=4, kv_heads=1, head_dim=64, rank=8, adapters=1)),
    (7, 37, dict(hidden=1024, heads=8, kv_heads=2, head_dim=128, rank=16, adapters=3, page=8)),
    (40, 150, dict(hidden=768, heads=12, kv_heads=12, head_dim=64, rank=64, adapters=20))])
def test_decode_steps_match_the_plain_form(example, batch, steps, sizes):
    error, us = example.run(batch, steps, **sizes)
    assert error < 2.0 ** -6
