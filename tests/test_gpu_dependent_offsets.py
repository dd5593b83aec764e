"""GPU tests of calls whose offsets the kernel before them in the stream writes.

A launch may start while that kernel still runs (programmatic dependent launch); it waits
for its end before it reads anything.  The writer here lets the next launch in at once,
has the old offsets in every SM's first-level cache, and writes the new ones 300 us later:
a read moved before the wait, or served from a copy made before the write, gives the old
rows.  Both sets of offsets are valid ones.
"""
import ctypes
import subprocess

import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg
import test_gpu_ragged as ragged
import test_gpu_w4 as w4

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32

WRITER = r"""
#include <cuda_runtime.h>
__device__ unsigned long long now() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// block 0 writes `from` to `to` 300 us after the start; every block has read `to` before
__global__ void writer(int *to, const int *from, int n, int *sink) {
    int sum = 0;
    for (int r = 0; r < 4; ++r)
        for (int i = threadIdx.x; i < n; i += blockDim.x) sum += __ldg(to + i) + *(volatile int *)(to + i);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned long long start = now();
    while (now() - start < 300000) {}
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < n; i += blockDim.x) to[i] = from[i];
    if (sum == -12345) *sink = sum;
}
extern "C" int launch_writer(int *to, const int *from, int n, int *sink, int blocks, void *stream) {
    writer<<<blocks, 32, 0, static_cast<cudaStream_t>(stream)>>>(to, from, n, sink);
    return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def launch_writer(tmp_path_factory):
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    folder = tmp_path_factory.mktemp("writer")
    (folder / "writer.cu").write_text(WRITER)
    subprocess.check_call([build.NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-shared",
                           "-Xcompiler", "-fPIC", "-o", str(folder / "writer.so"), str(folder / "writer.cu")])
    fn = ctypes.CDLL(str(folder / "writer.so")).launch_writer
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    sink = torch.zeros(1, dtype=torch.int32, device="cuda")
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count

    def launch(to, source):
        assert fn(to.data_ptr(), source.data_ptr(), to.numel(), sink.data_ptr(), blocks,
                  torch.cuda.current_stream().cuda_stream) == 0
    yield launch
    torch.cuda.synchronize()
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _follow(c, d, launch_writer, new):
    old, want = c.dev_off.clone(), torch.tensor(new, dtype=torch.int32, device="cuda")
    c.off = new
    for _ in range(10):
        c.dev_off.copy_(old)
        d.fill_(-77.0)
        torch.cuda.synchronize()
        launch_writer(c.dev_off, want)
        c.run(d)
        c.check(d, True)


@pytest.mark.parametrize("sizes,p,q", [([3, 5, 0, 8], 264, 136), ([300, 500, 0, 224], 2112, 520)])
@pytest.mark.parametrize("direction", [ragged.NT, ragged.NN, ragged.TN])
def test_ragged(launch_writer, direction, sizes, p, q):
    c = ragged.Case(direction, sizes, p, q, ints=True, seed=1)
    d = torch.empty((4, p, q) if direction == ragged.TN else (c.T, p if direction == ragged.NT else q),
                    dtype=F32 if direction == ragged.TN else BF16, device="cuda")
    T = c.T
    new = [0, T // 2, T // 2, T - 3, T]
    _follow(c, d, launch_writer, new)


@pytest.mark.parametrize("sizes", [[3, 5, 0, 8], [1] * 4])
def test_4_bit(launch_writer, sizes):
    c = w4.Case(sizes, 264, 640, 32, True, ints=True, seed=1)
    M = c.x.shape[0]
    d = torch.empty((M, 264), dtype=BF16, device="cuda")
    _follow(c, d, launch_writer, [0, M // 2, M // 2, M - 1, M])
