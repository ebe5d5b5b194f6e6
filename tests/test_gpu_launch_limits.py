"""GPU: kernels whose shared memory differs from call to call and from plan to plan, launched by several threads and after smaller plans
were made: no launch is refused, and results are those of one thread."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("mode", [dg.GEMM_SCALE_BLOCK_1x128_128x128, dg.GEMM_SCALE_MX_E8M0_32])
def test_a_plan_of_fewer_stages_leaves_a_deeper_one_running(mode):
    m, n, k = 512, 512, 2048
    a, b = (randn(r, k, seed=i).to(torch.float8_e4m3fn) for i, r in enumerate((m, n)))
    d = torch.empty(m, n, device="cuda")
    mx = mode == dg.GEMM_SCALE_MX_E8M0_32
    if mx:
        sa, sb = (torch.full((-(-r // 128) * -(-k // 128) * 512,), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    else:
        sa, sb = torch.ones(m, k // 128, device="cuda"), torch.ones(n // 128, k // 128, device="cuda")
    desc = lambda stages: dg.make_desc(m, n, k, dtype_a=dg.GEMM_E4M3, scale_mode=mode, stages=stages)  # noqa: E731

    def run(plan):
        d.fill_(float("nan"))
        if mx:
            plan.run_mx(a, b, d, sa, sb)
        else:
            plan.run(a, b, d, scale_a=sa, scale_b=sb)
        assert plan.sync_status()[0] == dg.GEMM_OK
        return d.clone()

    with dg.Plan(desc(0)) as deep:
        want = run(deep)
        with dg.Plan(desc(2)) as flat:
            assert flat.info.smem_bytes < deep.info.smem_bytes
            assert torch.equal(run(deep), want)
            assert torch.equal(run(flat), want)
            assert torch.equal(run(deep), want)


def test_threads_with_calls_of_many_sizes():
    sizes = [(t, n, k) for t in (1, 5, 8) for n, k in ((256, 512), (512, 4096), (300, 14336), (64, 28672))]
    work = []
    for i, (t, n, k) in enumerate(sizes):
        codes = torch.randint(0, 256, (n, k // 2), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda").to(torch.uint8)
        work.append((randn(t, k, seed=i), codes, (randn(n, k // 128, seed=i + 1) * 0.01)))
    norms = [(randn(t, n, seed=t), randn(t, n, seed=t + 1)) for t, n in ((3, 64), (40, 1000), (900, 4096), (300, 16384), (200, 20000))]

    def everything(order):
        out = {}
        for i in order:
            if i < len(work):
                out[i] = dg.int4_matmul(*work[i])
            else:
                x, r = norms[i - len(work)]
                out[i] = dg.add_rms_norm(x, residual=r)[0], dg.add_rms_norm_backward(x, r)[0]
        return out

    indices = list(range(len(work) + len(norms)))
    results, errors = [], []

    def worker(shift):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                got = everything(indices[shift:] + indices[:shift])
                torch.cuda.current_stream().synchronize()
            results.append(got)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=worker, args=(3 * s,)) for s in range(5)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    want = everything(indices)
    for got in results:
        for i in indices:
            pairs = zip(got[i], want[i]) if i >= len(work) else [(got[i], want[i])]
            assert all(torch.equal(a, b) for a, b in pairs), i


COLD = """
import torch
import dense_gemm_blackwell_gb300 as dg
dg.build()
torch.manual_seed(0)
bf16 = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
x, r, w = bf16(8, 8192), bf16(8, 8192), bf16(8192)
codes = torch.randint(0, 256, (512, 4096), device="cuda").to(torch.uint8)
scales, w2, out = bf16(512, 64) * 0.01, bf16(512, 8192) * 0.01, bf16(8, 256)
plan = dg.GatedPlan(8, 256, 8192)
torch.cuda.synchronize()
def step():
    n, s, h = dg.add_rms_norm(x, w, residual=r, scale_mode=dg.GEMM_SCALE_BLOCK_1x128_128x128)
    return s, h, *dg.add_rms_norm_backward(x, r, w), dg.int4_matmul(x, codes, scales), plan.run(x, w2, out)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = step()
graph.replay()
torch.cuda.synchronize()
captured = [t.clone() for t in captured]
assert all(torch.equal(a, b) for a, b in zip(captured, step()))
print("same")
"""


def test_first_calls_of_a_process_inside_a_capture():
    """What a kernel's first launch asks of the runtime may be asked while a graph is recorded."""
    done = subprocess.run([sys.executable, "-c", COLD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip().endswith("same"), done.stderr[-2000:]
