"""Timed cases of the expert operators that work on ragged groups and on 4-bit weights.

Every operator is here twice: in its plain form, elementary torch operations in
32 bits (``own`` false), and as the library's calls (``own`` true).

Operators (``op`` of a case):

* ``fwd``        expert products on sorted tokens, D[r] = A[r] W[g(r)]^T
* ``dgrad``      their input gradient, dA[r] = dD[r] W[g(r)]
* ``wgrad``      their weight gradient, dW[g] = sum over the rows r of g of dD[r]^T A[r]
* ``w4``         products of a few tokens with 4-bit weights, w = scale * (code - zero)
* ``w4_ragged``  the same grouped by expert, tokens sorted by expert

``rows`` is the length of the token buffer, ``tokens`` how many of its rows
belong to experts (the others lie behind the last expert and stay as they
are), ``skew`` the exponent of the experts' popularity (0: all alike).
"""
import math

import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # a prompt's tokens through the experts' first products (the library's contiguous benchmark, unpadded)
        dict(name="forward prompt", op="fwd", groups=4, rows=32768, tokens=32768, n=4096, k=7168, skew=0.0),
        # a batch of single tokens in 16 experts: the weights' bytes count
        dict(name="forward decode", op="fwd", groups=16, rows=64, tokens=64, n=4096, k=7168, skew=0.5),
        # many narrow experts, popularity far from even, some experts without a token, rows left over
        dict(name="forward many experts", op="fwd", groups=64, rows=4096, tokens=3999, n=1000, k=2112, skew=1.0),
        # the training step's gradients of the first case and of many narrow experts
        dict(name="dgrad prompt", op="dgrad", groups=4, rows=32768, tokens=32768, n=4096, k=7168, skew=0.0),
        dict(name="dgrad many experts", op="dgrad", groups=64, rows=4096, tokens=3999, n=1000, k=2112, skew=1.0),
        dict(name="wgrad prompt", op="wgrad", groups=4, rows=32768, tokens=32768, n=4096, k=7168, skew=0.0, out="fp32"),
        dict(name="wgrad many experts", op="wgrad", groups=64, rows=4096, tokens=3999, n=1000, k=2112, skew=1.0,
             out="bf16"),
        # one token through one projection: the smallest call, where latency counts
        dict(name="w4 one token", op="w4", m=1, n=4096, k=7168, group=128, zeros=False),
        # a small batch, short groups with zero points, an odd number of tokens
        dict(name="w4 batch", op="w4", m=13, n=7168, k=2048, group=32, zeros=True),
        # a wide projection
        dict(name="w4 wide", op="w4", m=8, n=16384, k=7168, group=64, zeros=False),
        # one token's eight experts out of 64
        dict(name="w4 eight experts", op="w4_ragged", groups=64, rows=8, tokens=8, n=4096, k=2048, skew=0.0, group=32,
             zeros=True),
        # a batch of single tokens in 16 experts
        dict(name="w4 decode", op="w4_ragged", groups=16, rows=64, tokens=64, n=4096, k=7168, skew=0.5, group=128,
             zeros=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step if step > 1 else int(v)))


def draw(rng):
    while True:
        op = rng.choice(["fwd", "dgrad", "wgrad", "w4", "w4_ragged"])
        if op in ("fwd", "dgrad", "wgrad"):
            c = dict(op=op, groups=_log(rng, 1, 64), rows=_log(rng, 1, 32768), n=_log(rng, 64, 8192, 8),
                     k=_log(rng, 64, 8192, 8), skew=rng.choice([0.0, 0.5, 1.0]))
            c["tokens"] = c["rows"] if rng.random() < 0.5 else rng.randint(0, c["rows"])
            if op == "wgrad":
                c["out"] = rng.choice(["fp32", "bf16"])
        else:
            group = rng.choice([32, 64, 128])
            c = dict(op=op, n=_log(rng, 256, 16384, 8), k=_log(rng, 512, 16384, group), group=group,
                     zeros=rng.random() < 0.5)
            if op == "w4":
                c["m"] = _log(rng, 1, 32)
            else:
                c.update(groups=_log(rng, 2, 64), rows=_log(rng, 1, 128), skew=rng.choice([0.0, 0.5, 1.0]))
                c["tokens"] = c["rows"] if rng.random() < 0.5 else rng.randint(0, c["rows"])
        weights = c.get("groups", 1) * c["n"] * c["k"]
        big = 4 * 4096 * 7168 * (4 if op in ("fwd", "dgrad") else 1)
        if c.get("tokens", 1) and weights <= big and c.get("rows", 0) * c["n"] * c["k"] <= 32768 * 4096 * 7168:
            return c


# ------------------------------------------------------------------ inputs
def _sizes(case, seed):
    """Rows of each expert, drawn by popularity; a host list, as the plain form splits by it."""
    g = torch.Generator().manual_seed(seed * 7 + 1)
    p = (1.0 + torch.arange(case["groups"], dtype=torch.float64)) ** -case["skew"]
    p = p[torch.randperm(case["groups"], generator=g)]
    ids = torch.multinomial(p / p.sum(), case["tokens"], replacement=True, generator=g)
    return torch.bincount(ids, minlength=case["groups"]).tolist()


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=BF16).mul_(scale)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    n, k = case["n"], case["k"]
    if "groups" in case:
        sizes = _sizes(case, seed)
        s["sizes"], s["used"] = sizes, case["tokens"]
        s["offsets"] = torch.tensor([sum(sizes[:i]) for i in range(len(sizes) + 1)], dtype=torch.int32, device="cuda")
    if case["op"] in ("fwd", "dgrad", "wgrad"):
        T, G = case["rows"], case["groups"]
        s["x"] = _normal(g, (T, k))
        s["dy"] = _normal(g, (T, n))
        if case["op"] == "wgrad":
            dtype = torch.float32 if case["out"] == "fp32" else BF16
            s["out"] = torch.zeros((G, n, k), dtype=dtype, device="cuda")
        else:
            s["w"] = _normal(g, (G, n, k), k ** -0.5)
            s["out"] = torch.zeros((T, n if case["op"] == "fwd" else k), dtype=BF16, device="cuda")
        return s
    G = case.get("groups", 1)
    lead = (G,) if "groups" in case else ()
    M, ng = case.get("rows", case.get("m")), k // case["group"]
    s["x"] = _normal(g, (M, k))
    # codes of bell-shaped weights, about 2.5 steps wide
    code = torch.randn(lead + (n, k), generator=g, device="cuda", dtype=BF16).mul_(2.5).round_().add_(8).clamp_(0, 15)
    code = code.to(torch.uint8).view(lead + (n, k // 2, 2))
    s["codes"] = code[..., 0] | (code[..., 1] << 4)
    s["scales"] = (torch.rand(lead + (ng, n), generator=g, device="cuda") * 0.75 + 0.25).mul_(k ** -0.5).to(BF16)
    s["zeros"] = (torch.randint(5, 12, lead + (ng, n), generator=g, device="cuda").to(torch.uint8)
                  if case["zeros"] else None)
    s["out"] = torch.zeros((M, n), dtype=BF16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def _weights32(codes, scales, zeros):
    """4-bit codes [n, k/2] with scales and zero points [k/group, n] as 32-bit weights [n, k]."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    q = q.unflatten(-1, (scales.shape[0], -1))
    z = 8.0 if zeros is None else zeros.t().float().unsqueeze(-1)
    return ((q - z) * scales.t().float().unsqueeze(-1)).flatten(-2)


def run(s):
    if own:
        return _run_own(s)
    op, out = s["op"], s["out"]
    if op == "w4":
        out.copy_(s["x"].float() @ _weights32(s["codes"], s["scales"], s["zeros"]).t())
        return out
    sizes, used = s["sizes"], s["used"]
    x = s["x"][:used].split(sizes)
    if op == "wgrad":
        dy = s["dy"][:used].split(sizes)
        [o.copy_(b.float().t() @ a.float()) for a, b, o in zip(x, dy, out)]
        return out
    into = out[:used].split(sizes)
    if op == "fwd":
        [o.copy_(a.float() @ w.float().t()) for a, w, o in zip(x, s["w"], into) if len(a)]
    elif op == "dgrad":
        dy = s["dy"][:used].split(sizes)
        [o.copy_(b.float() @ w.float()) for b, w, o in zip(dy, s["w"], into) if len(b)]
    else:
        zeros = [None] * len(sizes) if s["zeros"] is None else s["zeros"]
        [o.copy_(a.float() @ _weights32(c, sc, z).t())
         for a, c, sc, z, o in zip(x, s["codes"], s["scales"], zeros, into) if len(a)]
    return out


def _run_own(s):
    import moe_grouped_gemm_fp32_b200 as dg
    op, out = s["op"], s["out"]
    if op == "fwd":
        return dg.dg_m_grouped_bf16_gemm_nt_ragged(s["x"], s["w"], out, s["offsets"])
    if op == "dgrad":
        return dg.dg_m_grouped_bf16_gemm_nn_ragged(s["dy"], s["w"], out, s["offsets"])
    if op == "wgrad":
        return dg.dg_k_grouped_bf16_gemm_tn_ragged(s["dy"], s["x"], out, s["offsets"])
    if op == "w4":
        return dg.dg_w4_gemv_nt(s["x"], s["codes"], s["scales"], out, zeros=s["zeros"])
    return dg.dg_m_grouped_w4_gemv_nt_ragged(s["x"], s["codes"], s["scales"], out, s["offsets"], zeros=s["zeros"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    n, k = case["n"], case["k"]
    if case["op"] in ("fwd", "dgrad", "wgrad"):
        t, g = case["tokens"], case["groups"]
        if case["op"] == "wgrad":
            return {"bytes": 2 * t * (n + k) + g * n * k * (4 if case["out"] == "fp32" else 2), "flops": 2 * t * n * k}
        # every expert with a token has its weights read; by popularity most have one when tokens are many
        return {"bytes": 2 * t * (n + k) + 2 * _busy(case) * n * k, "flops": 2 * t * n * k}
    m = case.get("tokens", case.get("m"))
    per_expert = n * k // 2 + n * (k // case["group"]) * (3 if case["zeros"] else 2)
    return {"bytes": int(_busy(case) * per_expert) + 2 * m * (n + k), "flops": 2 * m * n * k}


def _busy(case):
    """Expected number of experts that have a token."""
    if "groups" not in case:
        return 1
    p = [(1.0 + i) ** -case["skew"] for i in range(case["groups"])]
    return sum(1 - (1 - q / sum(p)) ** case["tokens"] for q in p)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    out = s["out"].double()
    begin = 0
    if case["op"] == "w4":
        groups = [(0, slice(0, case["m"]))]
    else:
        groups = []
        for g, size in enumerate(s["sizes"]):
            groups.append((g, slice(begin, begin + size)))
            begin += size
    for g, rows in groups:
        x = s["x"][rows].double()
        if case["op"] == "fwd":
            out[rows] = torch.einsum("rk,nk->rn", x, s["w"][g].double())
        elif case["op"] == "dgrad":
            out[rows] = torch.einsum("rn,nk->rk", s["dy"][rows].double(), s["w"][g].double())
        elif case["op"] == "wgrad":
            out[g] = torch.einsum("rn,rk->nk", s["dy"][rows].double(), x)
        elif x.shape[0]:
            one = (lambda t: t) if case["op"] == "w4" else (lambda t: t[g])
            w = torch.empty((case["n"], case["k"]), dtype=torch.float64, device="cuda")
            byte = one(s["codes"])
            w[:, 0::2] = (byte % 16).double()
            w[:, 1::2] = (byte // 16).double()
            for j in range(case["k"] // case["group"]):
                col = slice(j * case["group"], (j + 1) * case["group"])
                zero = 8 if s["zeros"] is None else one(s["zeros"])[j].double()[:, None]
                w[:, col] = (w[:, col] - zero) * one(s["scales"])[j].double()[:, None]
            out[rows] = torch.einsum("rk,nk->rn", x, w)
    return out
