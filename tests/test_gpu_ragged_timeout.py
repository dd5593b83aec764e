"""Failure detection of the ragged BF16 products without a GPU fault.

A debug flag makes the producer warps issue no loads, so the bounded waits run
out (about 2 ms here).  The kernel must record DG_ERR_TIMEOUT in the device
status word and return, and the same call afterwards must be right.  Runs in a
child process because the wait limit is read once per process.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys, time
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
import moe_grouped_gemm_fp32_b200 as dg
from test_gpu_ragged import Case
dg.dg_get_device_status(clear=True)
for name, c in [("forward, thin", Case("nt", [3, 0, 5], 136, 264, ints=True)),
                ("input gradient", Case("nn", [70, 33], 136, 264, ints=True)),
                ("forward, pairs", Case("nt", [2100, 900, 3000], 2112, 520, ints=True)),
                ("weight gradient", Case("tn", [70, 33], 136, 264, ints=True)),
                ("weight gradient, single", Case("tn", [70, 33], 72, 264, ints=True))]:
    for dtype in ([torch.float32, torch.bfloat16] if c.dir == "tn" else [torch.bfloat16]):
        dg.dg_debug_set_flags(1)
        t0 = time.time()
        c.run(dtype=dtype)
        torch.cuda.synchronize()
        dt = time.time() - t0
        code = dg.dg_get_device_status(clear=True)
        assert code & 0xFF == 6, (name, hex(code))
        assert dt < 30, dt
        dg.dg_debug_set_flags(0)
        c.check(c.run(dtype=dtype), True)
        assert dg.dg_get_device_status(clear=True) == 0
        print(name, dtype, "timeout reported", hex(code), "in %.3f s; recovered" % dt)
print("OK")
"""


def test_bounded_waits_report_a_timeout_and_the_context_survives():
    env = dict(os.environ, DG_WAIT_TIMEOUT_CYCLES="4000000")
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "OK" in r.stdout
