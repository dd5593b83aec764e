"""GPU tests of the ragged and 4-bit products on ten streams at once, each stream
ordered behind the one that made its inputs and its result buffer."""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg
import test_gpu_ragged as ragged
import test_gpu_w4 as w4

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _ragged(direction, i):
    c = ragged.Case(direction, [300, 500], 520, 264, ints=True, seed=i)
    shape = (2, 520, 264) if direction == ragged.TN else (c.T, 520 if direction == ragged.NT else 264)
    return c, torch.full(shape, -77.0, dtype=F32 if direction == ragged.TN else BF16, device="cuda")


def _w4(sizes, i):
    c = w4.Case(sizes, 264, 4224, 32, True, ints=True, seed=i)
    return c, torch.full((c.x.shape[0], 264), -77.0, dtype=BF16, device="cuda")


@pytest.mark.parametrize("by_argument", [True, False])
def test_streams_at_once(by_argument):
    work = [_ragged(d, i) for i in range(2) for d in (ragged.NT, ragged.NN, ragged.TN)] + \
           [_w4(s, i) for i in range(2) for s in (5, [3, 4, 1, 0])]
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        for _, d in work:
            d.fill_(-77.0)
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for (c, d), s in zip(work, streams):
            if by_argument:
                c.run(d, stream=s)
            else:
                with torch.cuda.stream(s):
                    c.run(d)
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for c, d in work:
            c.check(d, True)
