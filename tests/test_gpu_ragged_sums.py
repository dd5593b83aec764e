"""GPU tests of the ragged BF16 products' sums over millions of products.

Operands lie in [1, 2), so all products have one sign and a sum that is cut off at
each step, not rounded, loses in proportion to its number of steps: the tensor
core adds 16 products at a time and cuts the partial sum, and one such sum of 2^24
products comes out 9.7 % low, 25 times a BF16 result's half step (2^-8).  Summed in FP32
over runs of 512 products (1024 for BF16 results), which are then added with rounding,
the bound is (run * 17 / 16 * 2^-23 + (runs + 2) * 2^-24) * S, with S the sum itself
here, and half a step of the result.
"""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _operand(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(shape, generator=g, device="cuda").add_(1).clamp_(max=1.9921875).to(BF16)


def _check(d, ref, count):
    run = 1024 if d.dtype == BF16 else 512
    sums = (run * 17 / 16 * 2.0 ** -23 + (count / run + 2) * 2.0 ** -24) * ref
    step = 2.0 ** -8 if d.dtype == BF16 else 2.0 ** -24
    err = (d.double() - ref).abs()
    assert (err <= step * (ref + sums) + sums).all(), float((err / ref).max())


def _product(a, b):
    """a [m, k] times b [n, k] in 64 bits, a piece of k at a time."""
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=F64, device="cuda")
    for k in range(0, a.shape[1], 1 << 20):
        out += a[:, k:k + (1 << 20)].double() @ b[:, k:k + (1 << 20)].double().t()
    return out


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_long_rows(direction, rows):
    K, N = 1 << 24, 8
    x, w = _operand((rows, K), 1), _operand((N, K), 2)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    d = torch.zeros((rows, N), dtype=BF16, device="cuda")
    if direction == "nt":
        dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w[None], d, off)
    else:
        dg.dg_m_grouped_bf16_gemm_nn_ragged(x, w.t().contiguous()[None], d, off)
    _check(d, _product(x, w), K)


@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_long_rows_on_cta_pairs(direction):
    K, N, rows = 1 << 20, 264, 2560                  # 20 pair tiles or more: as many as take pairs
    x, w = _operand((rows, K), 3), _operand((N, K), 4)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    d = torch.zeros((rows, N), dtype=BF16, device="cuda")
    if direction == "nt":
        dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w[None], d, off)
    else:
        dg.dg_m_grouped_bf16_gemm_nn_ragged(x, w.t().contiguous()[None], d, off)
    _check(d[::64], _product(x[::64], w), K)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N", [(8, 16), (136, 136)])
def test_many_tokens(M, N, dtype, accumulate):
    T = 1 << 24 if M == 8 else 1 << 22
    a, b = _operand((T, M), 5), _operand((T, N), 6)
    off = torch.tensor([0, T - 7], dtype=torch.int32, device="cuda")
    d = torch.zeros((1, M, N), dtype=dtype, device="cuda")
    dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, off, accumulate=accumulate)
    _check(d[0], _product(a[:T - 7].t(), b[:T - 7].t()), T)


@pytest.mark.parametrize("M,N", [(136, 264), (72, 264)])
@pytest.mark.parametrize("tokens", [8192, 8193])
def test_both_sides_of_one_level_sums(tokens, M, N):
    """BF16 weight gradients of up to 8192 tokens are summed in one level: at most
    tokens * 17 / 16 * 2^-23 of the sum, 1.1e-3, a quarter of the half step; more in two."""
    a, b = _operand((tokens, M), 7), _operand((tokens, N), 8)
    off = torch.tensor([0, 5, tokens], dtype=torch.int32, device="cuda")
    d = torch.zeros((2, M, N), dtype=BF16, device="cuda")
    dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, off)
    for g, (i, j) in enumerate([(0, 5), (5, tokens)]):
        ref = a[i:j].double().t() @ b[i:j].double()
        sums = tokens * 17 / 16 * 2.0 ** -23 * ref
        assert ((d[g].double() - ref).abs() <= 2.0 ** -8 * (ref + sums) + sums).all()
