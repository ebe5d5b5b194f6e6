"""GPU: a plan is ready for any stream when its creation returns.

The default stream is kept busy for some tenths of a second (a bounded delay) while plans are made and run on another
stream: what a plan's creation clears must not wait in the default stream's queue.  Before that, device memory that holds
no zeros is handed back to the driver, so that the plans' workspaces do not come zeroed by chance.
"""
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


def leave_dirty_memory():
    for size in (1 << 20, 1 << 24, 1 << 26):
        t = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
        del t
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def on_a_side_stream(work):
    """Runs `work` under a side stream while the default stream is busy, then waits for both."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    torch.cuda.synchronize()


def small_ints(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(256, 256, 16384), (300, 520, 4104)])
def test_product_with_split_tiles(M, N, K):
    a, b = small_ints(M, K, seed=1), small_ints(N, K, seed=2)
    want = (a.double() @ b.double().T).float()
    d = torch.full((2, M, N), float("nan"), device="cuda")
    leave_dirty_memory()
    plans = []

    def work():
        plans.append(dg.Plan(dg.make_desc(M, N, K)))
        for out in d:
            plans[0].run(a, b, out)
        assert plans[0].sync_status()[0] == dg.GEMM_OK

    on_a_side_stream(work)
    assert plans[0].info.stream_k_tiles > 0
    plans[0].close()
    assert torch.equal(d[0], want) and torch.equal(d[1], want)


def test_adapters_with_split_tiles():
    tokens, n, k, rank = 640, 512, 8192, 16
    x, w, a, b = small_ints(tokens, k, seed=3), small_ints(n, k, seed=4), small_ints(2, rank, k, seed=5), small_ints(2, n, rank, seed=6)
    x *= (torch.rand(tokens, k, device="cuda") < 0.02)               # keeps X A^T within 8 bits
    adapter = (torch.arange(tokens, device="cuda") % 3 - 1).to(torch.int32)
    t = x.double() @ a.double().flatten(0, 1).T
    assert t.abs().max() <= 256
    mine = adapter[:, None].long() == torch.arange(2, device="cuda")
    own = t.unflatten(1, (2, rank)) * mine[:, :, None]
    want = (x.double() @ w.double().T + torch.einsum("mir,inr->mn", own, b.double())).float()
    y = torch.full((2, tokens, n), float("nan"), device="cuda")
    leave_dirty_memory()
    plans = []

    def work():
        plans.append(dg.LoraPlan(tokens, n, k, rank=rank, adapters=2, dtype_y=dg.GEMM_F32))
        for out in y:
            plans[0].run(x, w, a, b, adapter, out)
        assert plans[0].sync_status()[0] == dg.GEMM_OK

    on_a_side_stream(work)
    assert plans[0].info.product.stream_k_tiles > 0
    plans[0].close()
    assert torch.equal(y[0], want) and torch.equal(y[1], want)


@pytest.mark.parametrize("length", [300, 20000])
def test_attention_with_split_sequences(length):
    """Values that are one in every element make the output one, whatever the probabilities are, if all parts are joined once."""
    pages = -(-length // 16)
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(2, 16, 128, generator=gen, device="cuda").to(torch.bfloat16)
    kc = torch.randn(2 * pages, 16, 2, 128, generator=gen, device="cuda").to(torch.bfloat16)
    vc = torch.ones_like(kc)
    table = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages)
    lengths = torch.tensor([length, length // 2], dtype=torch.int32, device="cuda")
    out = torch.full((2, 2, 16, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 2, 16), float("nan"), device="cuda")
    leave_dirty_memory()
    plans = []

    def work():
        plans.append(dg.PagedAttentionPlan(2, heads=16, kv_heads=2, head_dim=128, page_size=16))
        for o, s in zip(out, lse):
            plans[0].run(q, kc, vc, table, lengths, o, lse=s)

    on_a_side_stream(work)
    plans[0].run(q, kc, vc, table, lengths, out[0], lse=lse[0])        # the counters were left at zero
    torch.cuda.synchronize()
    plans[0].close()
    assert torch.equal(lse[0], lse[1]) and torch.isfinite(lse).all()
    # P is rounded to bf16 (2^-8 each) before its product with V, the sum of P is not
    assert ((out.float() - 1).abs() <= 2.0 ** -7).all() and torch.equal(out[0], out[1])
