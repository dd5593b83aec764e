"""GPU tests of how the ragged weight gradient ends an expert's tokens, and of its
bounded waits in calls that take longer than the bound.

Integers whose sums stay below 2^24 are exact in FP32, so an expert's result is equal
bit for bit to the exact one, rounded once, if and only if no token of a
neighbour (here NaN, or other integers) has reached it.
"""
import os
import subprocess
import sys

import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _problem(sizes, M, N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    make = lambda n: torch.randint(-3, 4, (off[-1], n), generator=g, device="cuda").to(BF16)
    return make(M), make(N), off


def _exact(a, b, off):
    return torch.stack([a[i:j].double().t() @ b[i:j].double() for i, j in zip(off, off[1:])])


# 136 x 136 and more: CTA pairs; the second CTA's columns of b exist or not
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("M,N", [(8, 8), (72, 200), (136, 136), (264, 520)])
def test_every_length_to_two_blocks(M, N, dtype):
    """Experts of 1 to 130 tokens, the last one ending with the buffer."""
    a, b, off = _problem(list(range(1, 131)), M, N)
    d = torch.full((130, M, N), float("nan"), dtype=dtype, device="cuda")
    dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, torch.tensor(off, dtype=torch.int32, device="cuda"))
    assert torch.equal(d, _exact(a, b, off).to(dtype))


@pytest.mark.parametrize("nan_in", ["a", "b", "both"])
@pytest.mark.parametrize("M,N", [(72, 200), (264, 520)])
def test_neighbours_of_nan(M, N, nan_in):
    """Every other expert's tokens are NaN: the ones between stay exact, call after call."""
    sizes = [1 + (7 * i) % 47 for i in range(300)]
    a, b, off = _problem(sizes, M, N, seed=1)
    want = _exact(a, b, off)[::2].to(F32)
    for g in range(1, len(sizes), 2):
        rows = slice(off[g], off[g + 1])
        if nan_in != "b":
            a[rows] = float("nan")
        if nan_in != "a":
            b[rows] = float("nan")
    dev = torch.tensor(off, dtype=torch.int32, device="cuda")
    d = torch.empty((len(sizes), M, N), dtype=F32, device="cuda")
    for _ in range(20):
        dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, dev)
        assert torch.equal(d[::2], want)
        assert d[1::2].isnan().all()


CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import moe_grouped_gemm_fp32_b200 as dg
BF16, F32 = torch.bfloat16, torch.float32
ones = lambda *s: torch.ones(s, dtype=BF16, device="cuda")
off = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")
dg.dg_get_device_status(clear=True)
L = 1 << 22
for M, N in ((8, 16), (136, 136)):
    for dtype in (F32, BF16):
        T = L + 5
        d = torch.zeros((1, M, N), dtype=dtype, device="cuda")
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a, b = ones(T, M), ones(T, N)
        t0.record()
        dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, off(T))
        t1.record()
        torch.cuda.synchronize()
        code = dg.dg_get_device_status(clear=True)
        print("weight gradient", M, N, dtype, "%.1f ms, status %x" % (t0.elapsed_time(t1), code))
        assert code == 0
        assert bool((d == torch.tensor(float(T)).to(dtype).item()).all())
        assert t0.elapsed_time(t1) > 3
for name, f, w in (("forward", dg.dg_m_grouped_bf16_gemm_nt_ragged, ones(1, 8, L)),
                   ("input gradient", dg.dg_m_grouped_bf16_gemm_nn_ragged, ones(1, L, 8))):
    d = torch.zeros((3, 8), dtype=BF16, device="cuda")
    x = ones(3, L)
    f(x, w, d, off(3))
    torch.cuda.synchronize()
    code = dg.dg_get_device_status(clear=True)
    print(name, "status %x" % code)
    assert code == 0 and bool((d == L).all())
d = torch.zeros((2560, 264), dtype=BF16, device="cuda")
x, w = ones(2560, L // 4), ones(264, L // 4)
for name, f, w in (("forward, pairs", dg.dg_m_grouped_bf16_gemm_nt_ragged, w[None]),
                   ("input gradient, pairs", dg.dg_m_grouped_bf16_gemm_nn_ragged, w.t().contiguous()[None])):
    d.zero_()
    f(x, w, d, off(2560))
    torch.cuda.synchronize()
    code = dg.dg_get_device_status(clear=True)
    print(name, "status %x" % code)
    assert code == 0 and bool((d == L // 4).all())
print("OK")
"""


def test_the_wait_limit_bounds_waits_not_calls():
    """Calls of several times the wait limit (4 million cycles, about 2 ms) end without
    a timeout: what a warp waits for at a time is short.  In a child process, as the
    limit is read once."""
    env = dict(os.environ, DG_WAIT_TIMEOUT_CYCLES="4000000")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=env, capture_output=True, text=True,
                       timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK" in r.stdout
