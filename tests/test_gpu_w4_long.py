"""GPU tests of the 4-bit products where a CTA goes through many chunks of K: scales, zero
points, x and the weights' slots are then filled again and again, and a stale one, or a
chunk out of order, shows in random operands.  (A chunk is 4 blocks of 128 k; the sizes
end inside a chunk, and some inside a block.)  Cases and tolerances: test_gpu_w4.py.
"""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg
from test_gpu_w4 import Case

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


# 97 blocks over 8 CTAs (12 or 13 each), 128 over 8, 41 over 8
@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("K,group,zeros", [(12320, 32, True), (12320, 32, False), (16384, 64, True), (16384, 128, False),
                                           (5248, 128, True)])
@pytest.mark.parametrize("M", [1, 13, 32])
def test_dense(M, K, group, zeros, ints):
    c = Case(M, 136, K, group, zeros, ints, seed=M + K)
    c.check(c.run(), ints)


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("K,group,zeros", [(12320, 32, True), (16384, 64, False), (16384, 128, True)])
@pytest.mark.parametrize("sizes", [[1], [0, 13, 2, 32], [5, 0, 40]])
def test_by_expert(sizes, K, group, zeros, ints):
    c = Case(sizes, 136, K, group, zeros, ints, lead=1, trail=2, seed=len(sizes) + K)
    c.check(c.run(), ints)


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("rows", [1, 5, 9])
def test_undivided(rows, group, zeros, ints):
    """Row blocks enough to fill the GPU: each CTA takes all of K, 19 blocks (18.75 in groups of 32)."""
    K = 2400 if group == 32 else 2432
    c = Case([rows] * 40, 2048, K, group, zeros, ints, seed=rows)
    c.check(c.run(), ints)
