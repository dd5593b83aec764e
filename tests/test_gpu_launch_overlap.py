"""GPU test of when a ragged product lets the next launch in.

A probe launched with programmatic stream serialisation behind the call takes the
time when it starts and again when the call before it is complete.  The call's
blocks may let it in while they wind down (microseconds), not while they still have
tiles to do (milliseconds here): blocks that come early crowd onto the SMs that
happen to be free.
"""
import ctypes
import subprocess

import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32

PROBE = r"""
#include <cuda_runtime.h>
__device__ unsigned long long now() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__global__ void probe(unsigned long long *out) {
    const unsigned long long start = now();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    out[0] = start;
    out[1] = now();
}
extern "C" int launch_probe(unsigned long long *out, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, probe, out);
}
"""


@pytest.fixture(scope="module")
def launch_probe(tmp_path_factory):
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    folder = tmp_path_factory.mktemp("probe")
    (folder / "probe.cu").write_text(PROBE)
    subprocess.check_call([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-shared",
                           "-Xcompiler", "-fPIC", "-o", str(folder / "probe.so"), str(folder / "probe.cu")])
    fn = ctypes.CDLL(str(folder / "probe.so")).launch_probe
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    return fn


def _call(name, L):
    z = lambda *s: torch.zeros(s, dtype=BF16, device="cuda")
    off = torch.tensor([0, 3 if name in ("nt", "nn") else L], dtype=torch.int32, device="cuda")
    if name == "nt":
        x, w, d = z(3, L), z(1, 8, L), z(3, 8)
        return lambda: dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w, d, off)
    if name == "nn":
        x, w, d = z(3, L), z(1, L, 8), z(3, 8)
        return lambda: dg.dg_m_grouped_bf16_gemm_nn_ragged(x, w, d, off)
    n = 8 if name == "tn" else 136                   # single CTA, CTA pair
    a, b, d = z(L, n), z(L, n), torch.zeros((1, n, n), dtype=F32, device="cuda")
    return lambda: dg.dg_k_grouped_bf16_gemm_tn_ragged(a, b, d, off)


@pytest.mark.parametrize("name", ["nt", "nn", "tn", "tn pair"])
def test_the_next_launch_starts_when_the_tiles_are_done(launch_probe, name):
    call = _call(name, 1 << 20)
    out = torch.zeros(2, dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        t0.record()
        call()
        t1.record()
        torch.cuda.synchronize()
        call()
        assert launch_probe(out.data_ptr(), stream) == 0
        torch.cuda.synchronize()
        took = t0.elapsed_time(t1) * 1e6
        start, end = out.tolist()
        assert took > 1e6, "one tile of a millisecond or more"
        assert end - start < took / 4, (end - start, took)
