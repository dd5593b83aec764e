"""Host-only checks (no GPU) of the ragged BF16 products and the 4-bit weight
products: the C entry points refuse bad arguments before any CUDA call, and the
binding passes sizes in the header's order and refuses buffers that disagree
with them."""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg
from moe_grouped_gemm_fp32_b200 import build as dg_build

FAKE = 0x10000   # a 16-byte aligned non-null address; never dereferenced on these paths
OK_BUT_NO_DEVICE = 4
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    dg_build.build()
    return dg.lib()


def _call(fn, base, **kw):
    args = dict(base)
    args.update(kw)
    return fn(*args.values(), None)


RAGGED = dict(a=FAKE, b=FAKE, d=FAKE, off=FAKE, M=64, N=256, K=512, G=4)


@pytest.mark.parametrize("name", ["dg_m_grouped_bf16_gemm_nt_ragged", "dg_m_grouped_bf16_gemm_nn_ragged"])
def test_m_grouped_refusals(L, name):
    f = getattr(L, name)
    for missing in ("a", "b", "d", "off"):
        assert _call(f, RAGGED, **{missing: None}) == 1
    for p in ("a", "b", "d"):
        assert _call(f, RAGGED, **{p: FAKE + 8}) == 2
    assert _call(f, RAGGED, M=-1) == 1
    assert _call(f, RAGGED, N=0) == 1
    assert _call(f, RAGGED, K=0) == 1
    assert _call(f, RAGGED, G=0) == 1
    assert _call(f, RAGGED, G=1025) == 3
    assert _call(f, RAGGED, N=252) == 3
    assert _call(f, RAGGED, K=516) == 3
    assert _call(f, RAGGED, M=(1 << 31) - 1, N=1 << 20) == 3      # more than 2^31 tiles
    assert _call(f, RAGGED, M=(1 << 31) - 1) == 3                 # a tile's last rows would pass 32 bits
    if not torch.cuda.is_available():
        assert _call(f, RAGGED) == OK_BUT_NO_DEVICE


WGRAD = dict(a=FAKE, b=FAKE, d=FAKE, f32=1, off=FAKE, G=4, M=256, N=128, K=64, acc=0)


def test_k_grouped_refusals(L):
    f = L.dg_k_grouped_bf16_gemm_tn_ragged
    for missing in ("a", "b", "d", "off"):
        assert _call(f, WGRAD, **{missing: None}) == 1
    for p in ("a", "b", "d"):
        assert _call(f, WGRAD, **{p: FAKE + 8}) == 2
    assert _call(f, WGRAD, K=-1) == 1
    assert _call(f, WGRAD, M=0) == 1
    assert _call(f, WGRAD, G=0) == 1
    assert _call(f, WGRAD, G=1025) == 3
    assert _call(f, WGRAD, M=260) == 3
    assert _call(f, WGRAD, N=130) == 3
    assert _call(f, WGRAD, G=1024, M=1 << 20, N=1 << 20) == 3
    assert _call(f, WGRAD, K=(1 << 31) - 1) == 3
    if not torch.cuda.is_available():
        assert _call(f, WGRAD) == OK_BUT_NO_DEVICE


W4 = dict(x=FAKE, w=FAKE, s=FAKE, z=None, d=FAKE, M=3, N=256, K=512, gs=128)
W4G = dict(x=FAKE, w=FAKE, s=FAKE, z=FAKE, d=FAKE, off=FAKE, M=3, N=256, K=512, G=8, gs=32)


def test_w4_refusals(L):
    for f, base in ((L.dg_w4_gemv_nt, W4), (L.dg_m_grouped_w4_gemv_nt_ragged, W4G)):
        for missing in ("x", "w", "s", "d"):
            assert _call(f, base, **{missing: None}) == 1
        for p in ("x", "w", "s", "z", "d"):
            assert _call(f, base, **{p: FAKE + 8}) == 2
        assert _call(f, base, M=-1) == 1
        assert _call(f, base, N=0) == 1
        assert _call(f, base, K=0) == 1
        assert _call(f, base, N=252) == 3
        assert _call(f, base, gs=16) == 3
        assert _call(f, base, gs=0) == 3
        assert _call(f, base, K=480, gs=64) == 3
        assert _call(f, base, N=65536 * 128) == 3
        assert _call(f, base, M=2000001) == 3
        if not torch.cuda.is_available():
            assert _call(f, base) == OK_BUT_NO_DEVICE
    assert _call(L.dg_m_grouped_w4_gemv_nt_ragged, W4G, off=None) == 1
    assert _call(L.dg_m_grouped_w4_gemv_nt_ragged, W4G, G=0) == 1
    assert _call(L.dg_m_grouped_w4_gemv_nt_ragged, W4G, G=1025) == 3


# ------------------------------------------------------------------ binding
class _FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("dg_"):
            raise AttributeError(name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def fake(monkeypatch):
    lib = _FakeLib()

    def req_cpu(t, dtype, name, ndim=None):
        # the real check minus "is on a CUDA device"
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if ndim is not None and t.dim() not in ((ndim,) if isinstance(ndim, int) else ndim):
            raise ValueError(f"{name} has {t.dim()} dims")
        return 0x1000
    monkeypatch.setattr(dg, "_req", req_cpu)
    monkeypatch.setattr(dg, "lib", lambda: lib)
    monkeypatch.setattr(dg, "_stream_handle", lambda stream: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return lib


def _ints(args):
    return [a for a in args if isinstance(a, int) and a != 0x1000]


def _z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_ragged_products(fake):
    off = _z(4, dtype=torch.int32)
    dg.dg_m_grouped_bf16_gemm_nt_ragged(_z(50, 40), _z(3, 24, 40), _z(50, 24), off)
    assert _ints(fake.calls[-1][1]) == [50, 24, 40, 3]
    dg.dg_m_grouped_bf16_gemm_nn_ragged(_z(50, 24), _z(3, 24, 40), _z(50, 40), off)
    assert _ints(fake.calls[-1][1]) == [50, 40, 24, 3]
    dg.dg_k_grouped_bf16_gemm_tn_ragged(_z(50, 24), _z(50, 40), _z(3, 24, 40, dtype=torch.float32), off, accumulate=True)
    assert _ints(fake.calls[-1][1]) == [1, 3, 24, 40, 50, 1]
    dg.dg_k_grouped_bf16_gemm_tn_ragged(_z(50, 24), _z(50, 40), _z(3, 24, 40), off)
    assert _ints(fake.calls[-1][1]) == [0, 3, 24, 40, 50, 0]
    with pytest.raises(ValueError, match="m_offsets"):
        dg.dg_m_grouped_bf16_gemm_nt_ragged(_z(50, 40), _z(3, 24, 40), _z(50, 24), off[:3].clone())
    with pytest.raises(ValueError, match="d has"):
        dg.dg_m_grouped_bf16_gemm_nt_ragged(_z(50, 40), _z(3, 24, 40), _z(49, 24), off)
    with pytest.raises(ValueError, match="b has"):
        dg.dg_m_grouped_bf16_gemm_nn_ragged(_z(50, 40), _z(3, 24, 40), _z(50, 40), off)
    with pytest.raises(ValueError, match="b has"):
        dg.dg_k_grouped_bf16_gemm_tn_ragged(_z(50, 24), _z(51, 40), _z(3, 24, 40), off)
    with pytest.raises(ValueError, match="d has"):
        dg.dg_k_grouped_bf16_gemm_tn_ragged(_z(50, 24), _z(50, 40), _z(2, 24, 40), off)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        dg.dg_k_grouped_bf16_gemm_tn_ragged(_z(50, 24), _z(50, 40), _z(3, 24, 40, dtype=torch.float16), off)
    with pytest.raises(ValueError, match="contiguous"):
        dg.dg_m_grouped_bf16_gemm_nt_ragged(_z(40, 50).t(), _z(3, 24, 40), _z(50, 24), off)


def test_binding_w4(fake):
    off = _z(4, dtype=torch.int32)
    u8 = torch.uint8
    dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 128, dtype=u8), _z(4, 24), _z(5, 24))
    assert _ints(fake.calls[-1][1]) == [5, 24, 256, 64]
    assert fake.calls[-1][1][3] is None                       # no zero points
    dg.dg_w4_gemv_nt(_z(5, 256), _z(1, 24, 128, dtype=u8), _z(1, 2, 24), _z(5, 24), zeros=_z(1, 2, 24, dtype=u8))
    assert _ints(fake.calls[-1][1]) == [5, 24, 256, 128]
    dg.dg_m_grouped_w4_gemv_nt_ragged(_z(5, 256), _z(3, 24, 128, dtype=u8), _z(3, 8, 24), _z(5, 24), off,
                                      zeros=_z(3, 8, 24, dtype=u8))
    assert _ints(fake.calls[-1][1]) == [5, 24, 256, 3, 32]
    with pytest.raises(ValueError, match="w has"):
        dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 64, dtype=u8), _z(4, 24), _z(5, 24))
    with pytest.raises(ValueError, match="w has"):
        dg.dg_w4_gemv_nt(_z(5, 257), _z(24, 128, dtype=u8), _z(4, 24), _z(5, 24))
    with pytest.raises(ValueError, match="scales has"):
        dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 128, dtype=u8), _z(4, 16), _z(5, 24))
    with pytest.raises(ValueError, match="zeros has"):
        dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 128, dtype=u8), _z(4, 24), _z(5, 24), zeros=_z(2, 24, dtype=u8))
    with pytest.raises(ValueError, match="d has"):
        dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 128, dtype=u8), _z(4, 24), _z(4, 24))
    with pytest.raises(ValueError, match="m_offsets"):
        dg.dg_m_grouped_w4_gemv_nt_ragged(_z(5, 256), _z(3, 24, 128, dtype=u8), _z(3, 8, 24), _z(5, 24),
                                          _z(3, dtype=torch.int32))


def test_binding_refuses_cpu_tensors():
    with pytest.raises(TypeError, match="CUDA"):
        dg.dg_w4_gemv_nt(_z(5, 256), _z(24, 128, dtype=torch.uint8), _z(4, 24), _z(5, 24))
    with pytest.raises(TypeError, match="CUDA"):
        dg.dg_m_grouped_bf16_gemm_nt_ragged(_z(50, 40), _z(3, 24, 40), _z(50, 24), _z(4, dtype=torch.int32))
