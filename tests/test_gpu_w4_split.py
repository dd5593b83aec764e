"""GPU test of how the 4-bit products divide K: by how the launch fills the GPU, so that
sizes next to one another are divided alike.  The choice is read from the launch line that
DG_VERBOSE prints, in a child process as the variable is read once."""
import os
import re
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
from moe_grouped_gemm_fp32_b200 import build
build.build()
import moe_grouped_gemm_fp32_b200 as dg
BF16 = torch.bfloat16
for K in {ks!r}:
    w = torch.full(({G}, {N}, K // 2), 0x99, dtype=torch.uint8, device="cuda")   # code 9: weight 1
    s = torch.ones(({G}, K // 128, {N}), dtype=BF16, device="cuda")
    x = torch.zeros(({M}, K), dtype=BF16, device="cuda")
    x[:, ::64] = 1
    off = torch.tensor([{M} * i // {G} for i in range({G} + 1)], dtype=torch.int32, device="cuda")
    d = torch.zeros(({M}, {N}), dtype=BF16, device="cuda")
    dg.dg_m_grouped_w4_gemv_nt_ragged(x, w, s, d, off)
    torch.cuda.synchronize()
    assert bool((d == K // 64).all())
assert dg.dg_get_device_status() == 0
"""


def _splits(ks, G, N, M):
    env = dict(os.environ, DG_VERBOSE="1")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, ks=list(ks), G=G, N=N, M=M)], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    got = [int(v) for v in re.findall(r"\[dg\] w4_gemv .*split=(\d+)", r.stderr)]
    assert len(got) == len(ks), r.stderr
    return got


def test_neighbouring_sizes_are_divided_alike():
    """16 experts of 32 row blocks: 512 CTAs leave some SMs with 4 and others with 3, whatever K is."""
    assert set(_splits([6144, 6912, 7040, 7168, 7296, 8192], 16, 4096, 64)) == {2}


def test_few_row_blocks_are_divided_most():
    assert _splits([7168], 1, 512, 1) == [8]


def test_many_row_blocks_stay_whole():
    assert _splits([1024], 16, 8192, 16) == [1]
