"""GPU tests of the ragged grouped BF16 products (forward, input gradient, weight
gradient) against their definition in 64 bits.

Tolerances.  Integer operands whose sums stay below 2^24 are exact in FP32, so
the result is the exact sum rounded once: equal bit for bit.  Real operands: a
BF16 result is off by at most half a step, eps / 2 = 2^-8 of the value; the
tensor core adds 16 products and the running sum, aligned to the largest and
truncated, so each of the K / 16 steps loses at most 17 * 2^-23 of the largest
partial sum, itself at most S = sum |a| |b|: K * 17 / 16 * 2^-23 * S.  FP32
weight gradients truncate over 512 tokens only and then round once per such
run: (512 * 17 / 16 * 2^-23 + runs * 2^-24) * S.
"""
import pytest
import torch

import moe_grouped_gemm_fp32_b200 as dg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NT, NN, TN = "nt", "nn", "tn"


@pytest.fixture(autouse=True, scope="module")
def _clean_status():
    from moe_grouped_gemm_fp32_b200 import build
    build.build()
    dg.dg_get_device_status(clear=True)
    yield
    assert dg.dg_get_device_status(clear=True) == 0, "a kernel recorded an error"


def _offsets(sizes, lead=0):
    o = [lead]
    for s in sizes:
        o.append(o[-1] + s)
    return o


def _dev(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


class Case:
    """Operands of one call; rows outside the offsets hold NaN."""

    def __init__(self, direction, sizes, p, q, lead=0, trail=0, ints=False, seed=0):
        # forward: p = N, q = K; dgrad: the same weights; wgrad: p = M, q = N
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dir, self.p, self.q, self.G = direction, p, q, len(sizes)
        self.off = _offsets(sizes, lead)
        self.T = self.off[-1] + trail
        make = (lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(BF16)) if ints else \
               (lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF16))
        self.x = make(self.T, q)
        self.y = make(self.T, p)
        self.w = make(self.G, p, q)
        inside = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        inside[self.off[0]:self.off[-1]] = True
        for t in (self.x, self.y):
            t[~inside] = float("nan")
        self.inside = inside
        self.dev_off = _dev(self.off)

    def rows(self):
        return [slice(a, b) for a, b in zip(self.off, self.off[1:])]

    def run(self, d=None, dtype=BF16, accumulate=False, stream=None):
        if self.dir == TN:
            if d is None:
                d = torch.full((self.G, self.p, self.q), float("nan"), dtype=dtype, device="cuda")
            return dg.dg_k_grouped_bf16_gemm_tn_ragged(self.y, self.x, d, self.dev_off, accumulate, stream=stream)
        if d is None:
            d = torch.full((self.T, self.p if self.dir == NT else self.q), -77.0, dtype=BF16, device="cuda")
        if self.dir == NT:
            return dg.dg_m_grouped_bf16_gemm_nt_ragged(self.x, self.w, d, self.dev_off, stream=stream)
        return dg.dg_m_grouped_bf16_gemm_nn_ragged(self.y, self.w, d, self.dev_off, stream=stream)

    def exact(self, absolute=False):
        v = (lambda t: t.double().abs()) if absolute else (lambda t: t.double())
        if self.dir == TN:
            return torch.stack([v(self.y[r]).t() @ v(self.x[r]) for r in self.rows()])
        out = torch.full((self.T, self.p if self.dir == NT else self.q), -77.0, dtype=F64, device="cuda")
        for g, r in enumerate(self.rows()):
            out[r] = v(self.x[r]) @ v(self.w[g]).t() if self.dir == NT else v(self.y[r]) @ v(self.w[g])
        return out

    def check(self, d, ints, base=None):
        torch.cuda.synchronize()
        ref = self.exact()
        if base is not None:
            ref = ref + base.double()
        if ints:
            assert ref.abs().max() < 2 ** 24
            assert torch.equal(d, ref.to(d.dtype)), float((d.double() - ref).abs().max())
            return
        s = self.exact(absolute=True)
        if base is not None:
            s = s + base.double().abs()
        tokens = max(b - a for a, b in zip(self.off, self.off[1:]))
        if self.dir != TN:
            k = self.q if self.dir == NT else self.p
            s = s * self.inside[:, None]
        else:
            k = tokens
        if d.dtype == F32:
            sums = (min(k, 512) * 17 / 16 * 2.0 ** -23 + (k / 512 + 2) * 2.0 ** -24) * s
            step = 2.0 ** -24
        else:
            sums = max(k, 16) * 17 / 16 * 2.0 ** -23 * s
            step = 2.0 ** -8
        err = (d.double() - ref).abs()
        assert torch.isfinite(err).all()
        bound = step * (ref.abs() + sums) + sums
        assert (err <= bound).all(), float((err / bound.clamp_min(1e-300)).max())


M_SIZES = [
    ([1], 0, 0),
    ([0, 5, 0], 3, 2),
    ([127, 1, 0, 129, 33], 1, 7),
    ([32, 31, 97, 64], 0, 0),
    ([128, 256, 300], 5, 60),            # CTA pairs
    ([0, 700, 1, 0, 257], 0, 300),       # CTA pairs: a group of one row, two empty ones
    ([3] * 70, 0, 1),                    # more groups than one set-up pass of 32
]


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("p,q", [(8, 8), (264, 136), (1000, 520), (72, 1032)])
@pytest.mark.parametrize("sizes,lead,trail", M_SIZES)
@pytest.mark.parametrize("direction", [NT, NN])
def test_m_grouped(direction, sizes, lead, trail, p, q, ints):
    c = Case(direction, sizes, p, q, lead, trail, ints, seed=len(sizes) + p)
    c.check(c.run(), ints)


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("sizes,lead,trail", [([0, 700, 1, 0, 257, 128, 1300], 3, 300), ([129, 2000, 127], 0, 0)])
@pytest.mark.parametrize("p,q", [(1032, 1064), (2112, 520), (520, 2112)])
@pytest.mark.parametrize("direction", [NT, NN])
def test_m_grouped_on_cta_pairs(direction, sizes, lead, trail, p, q, ints):
    """256-row tiles with runs that start, end and turn empty inside them."""
    c = Case(direction, sizes, p, q, lead, trail, ints, seed=len(sizes) + p)
    c.check(c.run(), ints)


K_SIZES = [
    ([1], 0, 0),
    ([0, 15, 16, 17, 0], 2, 5),
    ([63, 64, 65, 1, 48], 0, 9),
    ([513, 0, 1025, 7], 3, 0),
    ([2] * 40, 1, 1),
]


# few tiles of one expert in several row blocks; 128 rows by 64 and by 128 columns; 24
# rows on average by 128 columns, some experts with several row blocks or none
@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("sizes,lead,trail", [([256], 0, 0), ([257], 5, 40), ([33, 0, 95], 1, 2), ([100, 90, 129, 81], 3, 7),
                                              ([100] * 19 + [127], 0, 9), ([0, 20, 64, 31, 1, 33] * 4, 2, 30)])
@pytest.mark.parametrize("direction", [NT, NN])
def test_m_grouped_on_single_ctas(direction, sizes, lead, trail, ints):
    c = Case(direction, sizes, 1032, 1064, lead, trail, ints)
    c.check(c.run(), ints)


@pytest.mark.parametrize("ints", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,q", [(8, 8), (136, 264), (520, 1000), (264, 72)])
@pytest.mark.parametrize("sizes,lead,trail", K_SIZES)
def test_k_grouped(sizes, lead, trail, p, q, dtype, ints):
    c = Case(TN, sizes, p, q, lead, trail, ints, seed=len(sizes) + q)
    c.check(c.run(dtype=dtype), ints)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("p,q", [(136, 264), (8, 72)])
def test_k_grouped_accumulates(p, q, dtype):
    """Added once, in FP32: integers stay exact; an expert without tokens keeps its gradient."""
    c = Case(TN, [70, 0, 17], p, q, 1, 2, ints=True, seed=3)
    base = torch.randint(-40, 41, (3, p, q), device="cuda").to(dtype)
    d = c.run(base.clone(), accumulate=True)
    c.check(d, True, base=base)
    assert torch.equal(d[1], base[1])
    c.run(d, accumulate=False)                   # and overwritten without it
    c.check(d, True)
    assert not d[1].any()


def test_no_tokens():
    w = torch.zeros((3, 16, 24), dtype=BF16, device="cuda")
    off = _dev([0, 0, 0, 0])
    e = lambda n: torch.empty((0, n), dtype=BF16, device="cuda")
    dg.dg_m_grouped_bf16_gemm_nt_ragged(e(24), w, e(16), off)
    dg.dg_m_grouped_bf16_gemm_nn_ragged(e(16), w, e(24), off)
    d = torch.full((3, 16, 24), 5.0, dtype=F32, device="cuda")
    dg.dg_k_grouped_bf16_gemm_tn_ragged(e(16), e(24), d, off, accumulate=True)
    assert bool((d == 5).all())
    dg.dg_k_grouped_bf16_gemm_tn_ragged(e(16), e(24), d, off)
    assert not d.any()
    # tokens in the buffer, none in an expert
    c = Case(NT, [0, 0], 16, 24, lead=3, trail=9)
    assert bool((c.run() == -77).all())
    c = Case(TN, [0, 0], 16, 24, lead=3, trail=9)
    assert not c.run().any()


@pytest.mark.parametrize("direction,sizes,p,q", [(NT, [2100, 900, 3000], 2112, 520), (NN, [2100, 900, 3000], 520, 2112),
                                                 (NT, [40] * 24, 2112, 264), (NN, [40] * 24, 264, 2112)])
def test_m_grouped_many_waves(direction, sizes, p, q):
    """More tiles than resident CTAs (pairs and single CTAs): every tile once, over several raster bands."""
    c = Case(direction, sizes, p, q, 2, 3, ints=True, seed=9)
    c.check(c.run(), True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_k_grouped_many_waves(dtype):
    c = Case(TN, [130, 1, 0, 700, 65], 2600, 2112, 2, 3, ints=True, seed=9)
    c.check(c.run(dtype=dtype), True)


def test_long_sums_keep_fp32():
    """FP32 weight gradients over many tokens are as exact as rounded FP32 sums."""
    c = Case(TN, [20000, 12000], 264, 136, seed=4)
    d = c.run(dtype=F32).double()
    ref = c.exact()
    # random walk of n rounded adds: error about 2^-24 sqrt(n) of the result's own
    # root-mean-square; the truncated runs of 512 tokens add 32 steps of up to 2^-23
    # with one sign each.  1e-6 lies above both and far below one long truncated sum (2e-5)
    assert float((d - ref).norm() / ref.norm()) < 2e-6


def test_bit_identical_repeats():
    for c, kw in ((Case(NT, [300, 5, 200], 264, 520, seed=1), {}), (Case(NN, [300, 5, 200], 264, 520, seed=1), {}),
                  (Case(TN, [300, 5, 200], 264, 520, seed=1), {"dtype": F32})):
        first = c.run(**kw).clone()
        for _ in range(3):
            assert torch.equal(c.run(**kw), first)


@pytest.mark.parametrize("direction", [NT, NN, TN])
def test_graph_replay_with_new_offsets(direction):
    """Offsets are read on the device: a captured call follows them."""
    c = Case(direction, [100, 300, 20], 264, 136, trail=200, ints=True, seed=6)
    c.x.nan_to_num_(nan=1.0), c.y.nan_to_num_(nan=1.0)
    d = c.run(dtype=F32) if direction == TN else c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            c.run(d, dtype=d.dtype)
    torch.cuda.current_stream().wait_stream(s)
    for off in ([0, 1, 1, 620], [7, 400, 401, 620], [0, 0, 0, 0]):
        c.off = off
        c.dev_off.copy_(_dev(off))
        c.inside[:] = False
        c.inside[off[0]:off[-1]] = True
        d.fill_(-77.0)
        g.replay()
        c.check(d, True)


def test_two_streams_at_once():
    cases = [Case(NT, [300, 500], 520, 264, ints=True, seed=i) for i in range(2)] + \
            [Case(TN, [300, 500], 264, 520, ints=True, seed=i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [c.run(stream=s) for c, s in zip(cases, streams) for _ in range(1)]
    torch.cuda.synchronize()
    for c, d in zip(cases, outs):
        c.check(d, True)


@pytest.mark.parametrize("direction", [NT, NN, TN])
@pytest.mark.parametrize("raw,used", [([0, 90, 40, 200], [0, 90, 90, 200]), ([-5, 10, 400, 300], [0, 10, 250, 250]),
                                      ([0, 1 << 30, 3, -(1 << 31)], [0, 250, 250, 250])])
def test_bad_offsets_are_recorded_and_clamped(direction, raw, used):
    c = Case(direction, [100, 100, 50], 136, 72, ints=True, seed=2)
    dg.dg_get_device_status(clear=True)
    c.dev_off = _dev(raw)
    d = c.run()
    torch.cuda.synchronize()
    assert dg.dg_get_device_status(clear=True) & 0xFF == 1
    c.off = used
    c.check(d, True)


def test_gradients_are_the_differences_of_the_forward():
    """<c, f(a + da) - f(a)> = <input gradient, da>, and the same for the weights, in exact integers."""
    c = Case(NT, [70, 0, 33], 40, 24, ints=True, seed=8)
    da = torch.randint(-1, 2, c.x.shape, device="cuda").to(BF16)
    dw = torch.randint(-1, 2, c.w.shape, device="cuda").to(BF16)
    up = c.y                                        # the output's gradient
    f = lambda x, w: dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w, torch.empty_like(up), c.dev_off).double()
    gx = dg.dg_m_grouped_bf16_gemm_nn_ragged(up, c.w, torch.empty_like(c.x), c.dev_off).double()
    gw = dg.dg_k_grouped_bf16_gemm_tn_ragged(up, c.x, torch.empty(c.w.shape, dtype=F32, device="cuda"), c.dev_off).double()
    base = f(c.x, c.w)
    assert base.abs().max() <= 256                  # integers that BF16 holds
    assert float((up.double() * (f(c.x + da, c.w) - base)).sum()) == float((gx * da.double()).sum())
    assert float((up.double() * (f(c.x, c.w + dw) - base)).sum()) == float((gw * dw.double()).sum())


def test_a_layer_trains_as_in_64_bits():
    """Router sort, both expert products, SwiGLU between them, and back through all of them."""
    torch.manual_seed(0)
    tokens, H, I, G, topk = 150, 264, 136, 6, 2
    x = torch.randn(tokens, H, device="cuda", dtype=BF16)
    w1 = (torch.randn(G, 2 * I, H, device="cuda") * H ** -0.5).to(BF16)
    w2 = (torch.randn(G, H, I, device="cuda") * I ** -0.5).to(BF16)
    p, ids = torch.randn(tokens, G, device="cuda").softmax(-1).topk(topk)
    flat, order = ids.flatten().sort(stable=True)
    src = order // topk
    off = torch.searchsorted(flat, torch.arange(G + 1, device="cuda")).to(torch.int32)
    scale = p.flatten()[order, None]

    def act(h):
        gate, up = h.chunk(2, -1)
        return torch.nn.functional.silu(gate) * up

    # 64 bits, by autograd
    X, W1, W2 = (t.double().requires_grad_() for t in (x, w1, w2))
    rows = [slice(int(a), int(b)) for a, b in zip(off[:-1], off[1:])]
    xs = X[src]
    hs = torch.cat([xs[r] @ W1[g].t() for g, r in enumerate(rows)])
    ys = torch.cat([act(hs[r]) @ W2[g].t() for g, r in enumerate(rows)])
    out = torch.zeros(tokens, H, dtype=F64, device="cuda").index_add(0, src, ys * scale.double())
    up = torch.randn(tokens, H, device="cuda", dtype=BF16)
    out.backward(up.double())

    # the library's calls
    bf = lambda *s: torch.empty(s, device="cuda", dtype=BF16)
    n = tokens * topk
    xr = x[src].contiguous()
    h = dg.dg_m_grouped_bf16_gemm_nt_ragged(xr, w1, bf(n, 2 * I), off)
    h32 = h.float().requires_grad_()
    a32 = act(h32)
    a = a32.detach().to(BF16)
    y = dg.dg_m_grouped_bf16_gemm_nt_ragged(a, w2, bf(n, H), off)
    got = torch.zeros(tokens, H, device="cuda").index_add(0, src, y.float() * scale)
    dy = (up[src].float() * scale).to(BF16)
    da = dg.dg_m_grouped_bf16_gemm_nn_ragged(dy, w2, bf(n, I), off)
    dw2 = dg.dg_k_grouped_bf16_gemm_tn_ragged(dy, a, torch.empty(w2.shape, device="cuda", dtype=F32), off)
    a32.backward(da.float())
    dh = h32.grad.to(BF16)
    dx = dg.dg_m_grouped_bf16_gemm_nn_ragged(dh, w1, bf(n, H), off)
    dw1 = dg.dg_k_grouped_bf16_gemm_tn_ragged(dh, xr, torch.empty(w1.shape, device="cuda", dtype=F32), off)
    dx = torch.zeros(tokens, H, device="cuda").index_add(0, src, dx.float())
    # at most six BF16 roundings of 2^-8 lie between the inputs and any of these
    for name, g, e in (("out", got, out), ("dw2", dw2, W2.grad), ("dw1", dw1, W1.grad), ("dx", dx, X.grad)):
        rel = float((g.double() - e.detach()).norm() / e.detach().norm())
        assert rel <= 6 * 2.0 ** -8, (name, rel)


def test_large_offsets_pass_32_bits():
    """Rows whose element index passes 2^31."""
    n = 8 * 1024
    T = (1 << 31) // n + 300
    x = torch.zeros((T, 8), dtype=BF16, device="cuda")
    x[-260:] = torch.randint(-3, 4, (260, 8), device="cuda").to(BF16)
    w = torch.randint(-3, 4, (2, n, 8), device="cuda").to(BF16)
    d = torch.zeros((T, n), dtype=BF16, device="cuda")
    off = _dev([T - 260, T - 250, T])
    dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w, d, off)
    torch.cuda.synchronize()
    assert torch.equal(d[T - 260:T - 250], (x[T - 260:T - 250].double() @ w[0].double().t()).to(BF16))
    assert torch.equal(d[T - 250:], (x[T - 250:].double() @ w[1].double().t()).to(BF16))
    assert not d[T - 400:T - 260].any()


@pytest.mark.parametrize("graph", [False, True])
def test_dependent_calls_in_a_row(graph):
    """Each call reads what the one before it wrote, and writes what an earlier one
    read; launches that overlap must give what calls with a wait between them give."""
    torch.manual_seed(3)
    T, H, I, G = 96, 512, 1024, 6
    off = _dev([0, 20, 20, 50, 51, 90, 96])
    w1 = (torch.randn(G, I, H, device="cuda") * H ** -0.5).to(BF16)
    w2 = (torch.randn(G, H, I, device="cuda") * I ** -0.5).to(BF16)
    codes = torch.randint(0, 256, (H, H // 2), device="cuda").to(torch.uint8)
    scales = (torch.rand(H // 64, H, device="cuda") * 0.01).to(BF16)
    start = torch.randn(T, H, device="cuda", dtype=BF16)
    x, y, z = (torch.empty(T, n, device="cuda", dtype=BF16) for n in (H, I, H))
    dw = torch.empty(G, I, H, device="cuda", dtype=F32)

    def chain(wait):
        x.copy_(start)
        dw.zero_()
        for _ in range(8):
            dg.dg_m_grouped_bf16_gemm_nt_ragged(x, w1, y, off)
            wait()
            dg.dg_k_grouped_bf16_gemm_tn_ragged(y, x, dw, off, accumulate=True)
            wait()
            dg.dg_m_grouped_bf16_gemm_nt_ragged(y, w2, z, off)
            wait()
            dg.dg_w4_gemv_nt(z, codes, scales, x)
            wait()
            dg.dg_m_grouped_bf16_gemm_nn_ragged(y, w1, z, off)
            wait()
            x.add_(z)
            wait()

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in (x, y, z, dw)]
    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                chain(lambda: None)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(5):
        for t in (x, y, z, dw):
            t.fill_(float("nan"))
        g.replay() if graph else chain(lambda: None)
        torch.cuda.synchronize()
        for got, ref in zip((x, y, z, dw), want):
            assert torch.equal(got, ref)
