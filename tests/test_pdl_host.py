"""Host check of the kernels that may start before the kernel ahead of them ends: what that
kernel can write must not be read as read-only data (non-coherent loads may be moved before
the wait, or served from a copy made before the write)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_early_starting_kernels_make_no_read_only_loads():
    files = [f for f in glob.glob(os.path.join(ROOT, "moe_grouped_gemm_fp32_b200", "csrc", "*_kernel.cuh"))
             if "grid_dependency_wait()" in open(f).read()]
    assert len(files) >= 2
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert not re.search(r"__ldg\b|ld\.global\.nc|__restrict__", code), f
