"""GPU tests of the 4-bit products' zero points at the end of their range: 0..127 are
used as they are; a larger one is recorded as DG_ERR_INVALID_VALUE (code 1) in the
device status word, as offsets out of range are, and its low seven bits are used."""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(autouse=True)
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _problem(G, M, N, K, group):
    """Integers and unit scales: sums of |x| |q - z| stay below 2^24, so FP32 sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF16)
    w = torch.randint(0, 256, (G, N, K // 2), generator=g, device="cuda").to(torch.uint8)
    s = torch.ones((G, K // group, N), dtype=BF16, device="cuda")
    z = torch.randint(0, 128, (G, K // group, N), generator=g, device="cuda").to(torch.uint8)
    return x, w, s, z


def _exact(x, w, z, group):
    q = torch.stack((w & 15, w >> 4), dim=-1).flatten(-2).to(F64)
    return (x.to(F64) @ (q - z.to(F64).t().repeat_interleave(group, 1)).t()).to(BF16)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(136, 1152), (264, 8320)])
@pytest.mark.parametrize("M", [1, 12, 20])
def test_dense(M, N, K, group):
    x, w, s, z = (t if t.dim() == 2 else t[0] for t in _problem(1, M, N, K, group))
    run = lambda: dg.dg_w4_gemv_nt(x, w, s, torch.empty((M, N), dtype=BF16, device="cuda"), zeros=z)
    want = _exact(x, w, z, group)
    assert torch.equal(run(), want)
    assert dg.dg_get_device_status(clear=True) == 0
    for j, n in ((0, 0), (K // group - 1, N - 1), (K // group // 2, N // 2 + 1)):
        z[j, n] |= 128
        d = run()
        assert dg.dg_get_device_status(clear=True) & 0xFF == 1, (j, n)
        assert torch.equal(d, want)
        z[j, n] &= 127


def test_by_expert():
    x, w, s, z = _problem(4, 6, 136, 640, 64)
    off = torch.tensor([0, 2, 2, 5, 6], dtype=torch.int32, device="cuda")
    d = torch.empty((6, 136), dtype=BF16, device="cuda")
    run = lambda: dg.dg_m_grouped_w4_gemv_nt_ragged(x, w, s, d, off, zeros=z)
    want = torch.cat([_exact(x[a:b], w[g], z[g], 64) for g, (a, b) in enumerate([(0, 2), (2, 2), (2, 5), (5, 6)])])
    z[1, 3, 7] = 255                                  # an expert without rows: never read
    run()
    assert dg.dg_get_device_status(clear=True) == 0
    z[3, 9, 135] |= 128
    run()
    assert dg.dg_get_device_status(clear=True) & 0xFF == 1
    assert torch.equal(d, want)
