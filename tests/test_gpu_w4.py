"""GPU tests of the products with 4-bit weights (dense and grouped by expert over
ragged rows) against their definition in 64 bits.

Tolerances.  The result is BF16: off by at most half a step, eps / 2 = 2^-8 of
the value.  Below that, the products of a group are added on the tensor cores
(16 products and the running sum, truncated: at most 17 * 2^-23 of the partial
sum for each 16, so group * 17 / 16 * 2^-23), scaled and added with one rounding
per group, at most (groups + 8) * 2^-24: in all (group * 17 / 16 * 2 + groups +
8) * 2^-24 * S with S = sum |scale (q - z)| |x|.  With integers for x and
powers of two for the scales the FP32 sums are exact and the result is the
exact one rounded once.
"""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F64 = torch.bfloat16, torch.float64


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


class Case:
    def __init__(self, sizes, N, K, group, zeros, ints=False, lead=0, trail=0, seed=0):
        """sizes: rows of each expert, or a number for the dense call."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dense = isinstance(sizes, int)
        sizes = [sizes] if self.dense else sizes
        self.G, self.N, self.K, self.group = len(sizes), N, K, group
        self.off = [lead]
        for s in sizes:
            self.off.append(self.off[-1] + s)
        M = self.off[-1] + trail
        self.x = (torch.randint(-3, 4, (M, K), generator=g, device="cuda").to(BF16) if ints else
                  torch.randn((M, K), generator=g, device="cuda", dtype=BF16))
        self.x[:lead] = float("nan")
        self.x[self.off[-1]:] = float("nan")
        self.w = torch.randint(0, 256, (self.G, N, K // 2), generator=g, device="cuda").to(torch.uint8)
        ng = K // group
        s = torch.rand((self.G, ng, N), generator=g, device="cuda")
        self.s = (torch.exp2((s * 4).floor() - 2) if ints else s + 0.25).to(BF16)
        self.z = torch.randint(0, 17, (self.G, ng, N), generator=g, device="cuda").to(torch.uint8) if zeros else None
        self.dev_off = torch.tensor(self.off, dtype=torch.int32, device="cuda")

    def run(self, d=None, stream=None):
        if d is None:
            d = torch.full((self.x.shape[0], self.N), -77.0, dtype=BF16, device="cuda")
        if self.dense:
            one = lambda t: None if t is None else t[0]
            return dg.dg_w4_gemv_nt(self.x, one(self.w), one(self.s), d, zeros=one(self.z), stream=stream)
        return dg.dg_m_grouped_w4_gemv_nt_ragged(self.x, self.w, self.s, d, self.dev_off, zeros=self.z, stream=stream)

    def weights(self, g):
        q = torch.empty((self.N, self.K), dtype=F64, device="cuda")
        q[:, 0::2] = (self.w[g] & 15).double()
        q[:, 1::2] = (self.w[g] >> 4).double()
        z = torch.full_like(self.s[g], 8) if self.z is None else self.z[g]
        rep = lambda t: t.double().t().repeat_interleave(self.group, 1)
        return (q - rep(z)) * rep(self.s[g])

    def check(self, d, ints):
        torch.cuda.synchronize()
        ref = torch.full(d.shape, -77.0, dtype=F64, device="cuda")
        s = torch.zeros_like(ref)
        for g, (a, b) in enumerate(zip(self.off, self.off[1:])):
            if b > a:
                w = self.weights(g)
                ref[a:b] = self.x[a:b].double() @ w.t()
                s[a:b] = self.x[a:b].double().abs() @ w.abs().t()
        if ints:
            assert (s.max() * 4) < 2 ** 24           # multiples of a quarter
            assert torch.equal(d, ref.to(BF16)), float((d.double() - ref).abs().max())
            return
        sums = (self.group * 17 / 8 + self.K // self.group + 8) * 2.0 ** -24 * s
        err = (d.double() - ref).abs()
        assert torch.isfinite(err).all()
        bound = 2.0 ** -8 * (ref.abs() + sums) + sums
        assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(8, 128), (136, 640), (1000, 1152), (264, 4224)])
@pytest.mark.parametrize("M", [1, 7, 8, 9, 16, 17, 32, 33, 70])
def test_dense(M, N, K, group, zeros, ints):
    c = Case(M, N, K, group, zeros, ints, seed=M + N)
    c.check(c.run(), ints)


@pytest.mark.parametrize("K", [32, 96, 288, 480])
def test_short_k(K):
    """K that ends inside a stage, down to one group of 32."""
    c = Case(5, 72, K, 32, True, ints=True, seed=K)
    c.check(c.run(), True)


RAGGED = [
    ([1], 0, 0),
    ([0, 3, 0, 1], 2, 1),
    ([9, 0, 20, 1, 40], 0, 5),
    ([1] * 40, 1, 0),
    ([0, 0, 100], 0, 0),
]


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("N,K", [(136, 640), (264, 2176)])
@pytest.mark.parametrize("sizes,lead,trail", RAGGED)
def test_ragged(sizes, lead, trail, N, K, group, zeros, ints):
    c = Case(sizes, N, K, group, zeros, ints, lead, trail, seed=len(sizes) + N)
    c.check(c.run(), ints)


def test_all_codes_and_zero_points():
    """Every code against every zero point, one at a time: exact."""
    N, K = 128, 512                                   # row n: zero point n; x picks one k per token
    w = torch.arange(16, device="cuda").repeat(N, K // 16)
    packed = (w[:, 0::2] | (w[:, 1::2] << 4)).to(torch.uint8)
    z = torch.arange(N, device="cuda").to(torch.uint8)[None].repeat(K // 32, 1)
    s = torch.ones((K // 32, N), dtype=BF16, device="cuda")
    x = torch.zeros((16, K), dtype=BF16, device="cuda")
    x[torch.arange(16), torch.arange(16) * 17] = 1.0
    d = dg.dg_w4_gemv_nt(x, packed, s, torch.empty((16, N), dtype=BF16, device="cuda"), zeros=z)
    q = w[0, torch.arange(16, device="cuda") * 17]
    assert torch.equal(d.long(), q[:, None] - torch.arange(N, device="cuda")[None])


def test_infinite_and_nan_rows_stay_in_their_rows():
    c = Case(6, 136, 640, 64, True, ints=True, seed=5)
    good = c.run().clone()
    c.x[2, 5] = float("nan")
    c.x[4, 600] = float("inf")
    d = c.run()
    rows = [0, 1, 3, 5]
    assert torch.equal(d[rows], good[rows])
    assert d[2].isnan().all() and not d[4].isfinite().any()


def test_no_rows():
    c = Case(0, 136, 640, 64, False)
    assert c.run().shape == (0, 136)
    c = Case([0, 0, 0], 136, 640, 64, False, lead=3, trail=2)
    assert bool((c.run() == -77).all())


def test_bit_identical_repeats():
    for c in (Case(3, 264, 4224, 32, True, seed=1), Case([1, 0, 12, 3], 264, 4224, 128, False, seed=1)):
        first = c.run().clone()
        for _ in range(3):
            assert torch.equal(c.run(), first)


def test_graph_replay_with_new_offsets():
    c = Case([3, 4, 1, 0], 264, 640, 32, True, ints=True, trail=4, seed=6)
    c.x.nan_to_num_(nan=1.0)
    d = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            c.run(d)
    torch.cuda.current_stream().wait_stream(s)
    for off in ([0, 0, 12, 12, 12], [1, 2, 2, 3, 11], [0, 0, 0, 0, 0]):
        c.off = off
        c.dev_off.copy_(torch.tensor(off, dtype=torch.int32))
        d.fill_(-77.0)
        g.replay()
        c.check(d, True)


def test_streams_at_once():
    cases = [Case([3, 4, 1, 0], 264, 4224, 32, True, ints=True, seed=i) for i in range(3)]
    torch.cuda.synchronize()
    outs = [c.run(stream=torch.cuda.Stream()) for c in cases]
    torch.cuda.synchronize()
    for c, d in zip(cases, outs):
        c.check(d, True)


@pytest.mark.parametrize("raw,used", [([0, 9, 4, 20], [0, 9, 9, 20]), ([-5, 1, 40, 30], [0, 1, 25, 25]),
                                      ([0, 1 << 30, 3, -(1 << 31)], [0, 25, 25, 25])])
def test_bad_offsets_are_recorded_and_clamped(raw, used):
    c = Case([10, 10, 5], 136, 640, 64, False, ints=True, seed=2)
    dg.dg_get_device_status(clear=True)
    c.dev_off = torch.tensor(raw, dtype=torch.int32, device="cuda")
    d = c.run()
    torch.cuda.synchronize()
    assert dg.dg_get_device_status(clear=True) & 0xFF == 1
    c.off = used
    c.check(d, True)


def test_weights_past_32_bits():
    """An expert whose weights' bytes start beyond 2^31."""
    N, K, G = 16384, 4096, 66
    w = torch.zeros((G, N, K // 2), dtype=torch.uint8, device="cuda")
    w[-1] = 0x99                                       # code 9: weight 1 * scale
    s = torch.ones((G, K // 128, N), dtype=BF16, device="cuda")
    x = torch.zeros((2, K), dtype=BF16, device="cuda")
    x[1, :7] = 1.0
    off = torch.tensor([0] * (G - 1) + [0, 2], dtype=torch.int32, device="cuda")
    d = dg.dg_m_grouped_w4_gemv_nt_ragged(x, w, s, torch.full((2, N), -1.0, dtype=BF16, device="cuda"), off)
    assert bool((d[0] == 0).all()) and bool((d[1] == 7).all())


def test_decode_follows_the_prompts_products():
    """The same sorted tokens through the BF16 experts and through their 4-bit copy."""
    c = Case([2, 0, 5, 1], 264, 640, 64, True, seed=7)
    w = torch.stack([c.weights(g) for g in range(c.G)])
    full = dg.dg_m_grouped_bf16_gemm_nt_ragged(c.x, w.to(BF16), torch.empty((8, 264), dtype=BF16, device="cuda"), c.dev_off)
    four = c.run()
    c.check(four, False)
    # the BF16 copy rounds each weight at 2^-8 and both results round at 2^-8
    s = torch.cat([c.x[a:b].double().abs() @ w[g].abs().t() for g, (a, b) in enumerate(zip(c.off, c.off[1:]))])
    err = (full.double() - four.double()).abs()
    assert (err <= 2.0 ** -8 * (s + 2 * full.double().abs()) + 640 * 2.0 ** -22 * s).all()
