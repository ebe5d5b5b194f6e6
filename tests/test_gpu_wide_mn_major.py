"""GPU: 512-wide tiles with MN-major operands, on request: bit-exact on integers, on SM pairs and single SMs, with halves that are split
and that are not, ragged edges and groups of 64 that M or N ends in."""
import pytest
import torch

import dense_gemm_blackwell_gb300 as dg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    dg.build()
    torch.cuda.init()


@pytest.mark.parametrize("flags", [dg.GEMM_FLAG_CTA_GROUP_1, dg.GEMM_FLAG_CTA_GROUP_2])
@pytest.mark.parametrize("mn_a,mn_b", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("m,n,k,ctas", [(512, 1024, 2048, 0), (600, 1096, 200, 0), (1024, 1536, 1600, 6), (256, 512, 64, 0), (320, 576, 4096, 4)])
def test_bit_exact(m, n, k, ctas, mn_a, mn_b, flags):
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    ints = lambda r, c: torch.randint(-4, 5, (r, -(-c // 8) * 8), generator=gen, device="cuda").to(torch.bfloat16)[:, :c]  # noqa: E731
    a, b = ints(k, m) if mn_a else ints(m, k), ints(k, n) if mn_b else ints(n, k)
    want = (a.T if mn_a else a).double() @ (b if mn_b else b.T).double()
    d = torch.full((m, n), float("nan"), device="cuda")
    desc = dg.make_desc(m, n, k, major_a=mn_a, major_b=mn_b, lda=a.stride(0), ldb=b.stride(0), flags=flags, tile_n=512, max_ctas=ctas)
    with dg.Plan(desc) as plan:
        for _ in range(2):
            d.fill_(float("nan"))
            plan.run(a, b, d)
            assert plan.sync_status()[0] == dg.GEMM_OK
            assert plan.info.tile_n == 512
            assert torch.equal(d.double(), want)


@pytest.mark.parametrize("m,n,k", [(640, 704, 200), (1024, 512, 4096), (200, 136, 96)])
def test_groups_and_boxes_give_the_same_bits(m, n, k):
    """M and N of whole groups of 64 take one box a stage; the same columns of a wider matrix two."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    a, b = (torch.randn(k, c + 8, generator=gen, device="cuda").to(torch.bfloat16) for c in (m, n))
    out = []
    for extra in (0, 8):
        d = torch.full((m + extra, n + extra), float("nan"), device="cuda")
        desc = dg.make_desc(m + extra, n + extra, k, major_a=1, major_b=1, lda=m + 8, ldb=n + 8, tile_n=128,
                            flags=dg.GEMM_FLAG_CTA_GROUP_1 | dg.GEMM_FLAG_NO_STREAM_K)
        with dg.Plan(desc) as plan:
            plan.run(a, b, d)
            assert plan.sync_status()[0] == dg.GEMM_OK
        out.append(d[:m, :n])
    assert torch.equal(out[0], out[1])
    assert (out[0].double() - a[:, :m].double().T @ b[:, :n].double()).abs().max() < 1e-2


def test_groups_and_boxes_of_a_short_k():
    test_groups_and_boxes_give_the_same_bits(192, 128, 96)


@pytest.mark.parametrize("flags", [dg.GEMM_FLAG_CTA_GROUP_1, dg.GEMM_FLAG_CTA_GROUP_2])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k,ctas", [(512, 1024, 2048, 0), (600, 1096, 200, 0), (1024, 1536, 1600, 6)])
def test_16_bit_outputs(m, n, k, ctas, kind, flags):
    """Integers' products are exact in fp32 and rounded once."""
    gen = torch.Generator(device="cuda").manual_seed(m + n + k + 1)
    a, b = (torch.randint(-4, 5, (k, c), generator=gen, device="cuda").to(kind) for c in (m, n))
    want = (a.double().T @ b.double()).to(kind)
    code = dg.GEMM_BF16 if kind == torch.bfloat16 else dg.GEMM_F16
    d = torch.full((m, n), float("nan"), dtype=kind, device="cuda")
    desc = dg.make_desc(m, n, k, dtype_a=code, dtype_d=code, major_a=1, major_b=1, flags=flags, tile_n=512, max_ctas=ctas)
    with dg.Plan(desc) as plan:
        plan.run(a, b, d)
        assert plan.sync_status()[0] == dg.GEMM_OK
        assert plan.info.tile_n == 512 and torch.equal(d, want)
