"""GPU tests that name the kernel instantiation they are meant for.

The host chooses tiles by sizes, so a case meant for one of them can come to lie on the
other side of a threshold.  Here each case states the launch that it expects (the line
that DG_VERBOSE prints) and is checked bit for bit on integers; in a child process, as the
variable is read once."""
import os
import re
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

THIN = "rows=32 bn={} .*ctas/mma=1"
WIDE = "rows=128 bn={} .*ctas/mma=1"
PAIR = "bn=256 .*ctas/mma=2"

# sizes, p, q, lead, trail, launch: forward p = N, q = K; input gradient p = K, q = N
M_CASES = [
    # a few rows an expert: thin tiles, 64 and 128 columns
    ([3], 264, 264, 0, 2, THIN.format(64)),
    ([3] * 70, 1032, 1032, 0, 1, THIN.format(128)),
    # up to 24 on average, some with a second row block, with 32 columns of the MMA, with rows
    # 16..31 of the second half of the epilogue warps, or with none
    ([0, 20, 60, 31, 1, 23] * 4, 1032, 1064, 2, 30, THIN.format(128)),
    ([32, 17, 16, 33, 0, 24, 48] * 4, 1064, 1032, 0, 0, THIN.format(128)),
    # one expert, few tiles: two row blocks, and 17 (raster bands of 9 and 8)
    ([60], 1032, 1064, 1, 3, THIN.format(64)),
    ([540], 504, 504, 0, 0, THIN.format(64)),
    # 128 rows, 64 and 128 columns; 17 row blocks and another expert
    ([100, 90, 129, 81], 1032, 1064, 3, 7, WIDE.format(64)),
    ([2170, 0, 300], 128, 128, 2, 4, WIDE.format(64)),
    ([100] * 19 + [127], 1032, 1064, 0, 9, WIDE.format(128)),
    # pairs: 17 row blocks (bands of 9 and 8), 33 (11 each), other experts around them
    ([4300, 700], 2112, 2112, 2, 3, PAIR),
    ([129, 8300, 2, 500], 520, 520, 0, 0, PAIR),
]
# sizes, p = M, q = N, dtype, launch
K_CASES = [
    ([63, 0, 70], 72, 264, "float32", "dir=2 rows=128 bn=128 .*f32=1 levels=2"),
    ([63, 0, 70], 72, 264, "bfloat16", "dir=2 rows=128 bn=128 .*f32=0 levels=1"),
    ([9000, 70], 72, 264, "bfloat16", "dir=2 rows=128 bn=128 .*f32=0 levels=2"),
    # 17 row blocks of 256 (bands of 9 and 8), two experts and more
    ([63, 0, 70], 4200, 520, "float32", "dir=2 .*bn=256 .*ctas/mma=2 f32=1 levels=2"),
    ([63, 0, 70], 4200, 520, "bfloat16", "dir=2 .*bn=256 .*ctas/mma=2 f32=0 levels=1"),
    ([9000, 1, 70], 4200, 520, "bfloat16", "dir=2 .*bn=256 .*ctas/mma=2 f32=0 levels=2"),
]
# sizes (a number: dense), N, K, group, zeros, launch
W4_CASES = [
    (1, 136, 12320, 32, True, "tokens=8 split=8 .*bufs=2"),
    (13, 136, 16384, 64, False, "tokens=16 split=8 .*bufs=2"),
    (32, 136, 16384, 128, True, "tokens=32 split=8 .*bufs=2"),
    ([5] * 40, 2048, 2400, 32, True, "tokens=16 split=1 .*bufs=2"),
    ([1] * 40, 2048, 2432, 128, False, "tokens=8 split=1 .*bufs=2"),
    ([0, 30, 3], 136, 640, 64, True, "tokens=32 split=2 .*bufs=1"),
]

CHILD = r"""
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
from moe_grouped_gemm_fp32_b200 import build
build.build()
import moe_grouped_gemm_fp32_b200 as dg
import test_gpu_ragged, test_gpu_w4
dg.dg_get_device_status(clear=True)
kind, cases = {kind!r}, {cases!r}
for i, c in enumerate(cases):
    if kind == "w4":
        case = test_gpu_w4.Case(c[0], c[1], c[2], c[3], c[4], ints=True, seed=i)
        case.check(case.run(), True)
    elif kind == "tn":
        case = test_gpu_ragged.Case("tn", c[0], c[1], c[2], 1, 2, ints=True, seed=i)
        case.check(case.run(dtype=getattr(torch, c[3])), True)
    else:
        case = test_gpu_ragged.Case(kind, c[0], c[1], c[2], c[3], c[4], ints=True, seed=i)
        case.check(case.run(), True)
assert dg.dg_get_device_status(clear=True) == 0
"""


@pytest.mark.parametrize("kind,cases", [("nt", M_CASES), ("nn", M_CASES), ("tn", K_CASES), ("w4", W4_CASES)])
def test_cases_take_the_launch_they_are_meant_for(kind, cases):
    env = dict(os.environ, DG_VERBOSE="1")
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), kind=kind, cases=cases)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    launches = re.findall(r"\[dg\] (?:ragged|w4_gemv) .*", r.stderr)
    assert len(launches) == len(cases), r.stderr
    for line, case in zip(launches, cases):
        assert re.search(case[-1], line), (line, case)
