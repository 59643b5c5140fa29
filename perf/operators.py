"""Cases for the operators that use quantised weights: products with 4-bit
codes and group scales in both directions, a mixture-of-experts layer over
such codes, and the layer norm around them.

``run`` is one pass: with ``own`` false from elementary torch operations in
fp32, rounded once at the end; with ``own`` true through the framework's entry
points.  ``exact`` is the same pass from the definition in fp64.
"""

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def listed():
    return [
        # one new token through a small layer: latency is all that counts
        dict(name="linear_1_1024x1024", op="linear", T=1, m=1024, n=1024, group=128, asym=False, dtype="bf16"),
        # one new token through the largest square layer, per-group symmetric grid
        dict(name="linear_1_8192x8192", op="linear", T=1, m=8192, n=8192, group=128, asym=False, dtype="bf16"),
        # a few tokens, odd sizes, fine groups with zero points, fp32 activations (the solver's own type)
        dict(name="linear_7_1000x1111_fp32", op="linear", T=7, m=1000, n=1111, group=32, asym=True, dtype="fp32"),
        # a batch of sequences decoding through an MLP projection
        dict(name="linear_48_14336x4096", op="linear", T=48, m=14336, n=4096, group=64, asym=True, dtype="fp16"),
        # a prompt or a calibration batch through the largest square layer
        dict(name="linear_2048_8192x8192", op="linear", T=2048, m=8192, n=8192, group=128, asym=False, dtype="bf16"),
        # a tuning batch's gradient through the frozen MLP projection
        dict(name="grad_2048_4096x14336", op="grad", T=2048, m=4096, n=14336, group=128, asym=True, dtype="bf16"),
        # gradient samples for the Kronecker factors in fp32, odd sizes, one scale per row
        dict(name="grad_333_1000x1300_fp32", op="grad", T=333, m=1000, n=1300, group=0, asym=False, dtype="fp32"),
        # one new token, many small experts
        dict(name="moe_1_e32k4_1024x704", op="moe", T=1, E=32, k=4, d=1024, f=704, group=64, asym=False, dtype="bf16"),
        # a few sequences decoding, a few wide experts (the 4096 x 14336 MLP shape)
        dict(name="moe_16_e8k2_4096x14336", op="moe", T=16, E=8, k=2, d=4096, f=14336, group=128, asym=False,
             dtype="bf16"),
        # one training pass of the norm: a few odd rows in fp32
        dict(name="norm_37_1111_fp32", op="norm", T=37, d=1111, dtype="fp32"),
        # one training pass of the norm over a calibration batch
        dict(name="norm_8192_4096", op="norm", T=8192, d=4096, dtype="bf16"),
        # the widest rows
        dict(name="norm_2048_14336_fp16", op="norm", T=2048, d=14336, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.4:   # real layers are mostly multiples of 64, some sizes are odd
        return max(lo, min(hi, v))
    return max(lo, min(hi, max(64, v // 64 * 64) if hi >= 64 and v >= 64 else v))


def draw(rng):
    op = rng.choice(["linear", "linear", "grad", "moe", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    asym = rng.random() < 0.5
    group = rng.choice([0, 32, 64, 96, 128, 128, 256])
    while True:
        if op == "linear":
            c = dict(op=op, T=_log(rng, 1, 2048), m=_log(rng, 100, 14336), n=_log(rng, 100, 14336),
                     group=group, asym=asym, dtype=dtype)
        elif op == "grad":
            c = dict(op=op, T=_log(rng, 32, 2048), m=_log(rng, 100, 14336), n=_log(rng, 100, 14336),
                     group=group, asym=asym, dtype=dtype)
        elif op == "moe":
            E = rng.choice([4, 8, 16, 32, 60])
            c = dict(op=op, T=_log(rng, 1, 32), E=E, k=min(E, rng.choice([1, 2, 4, 6])), d=_log(rng, 256, 4096),
                     f=_log(rng, 256, 4096), group=group, asym=asym, dtype=dtype)
        else:
            c = dict(op=op, T=_log(rng, 1, 8192), d=_log(rng, 64, 14336), dtype=dtype)
        if 3072 in c.values():
            continue
        if op in ("linear", "grad") and c["T"] * c["m"] * c["n"] > 2048 * 8192 * 8192 // (4 if dtype == "fp32" else 1):
            continue
        if op == "moe" and c["E"] * c["d"] * c["f"] > 8 * 4096 * 14336:
            continue
        return c


# ---------------------------------------------------------------- inputs

def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + k)


def _groups(n, group):
    return 1 if not group or group >= n else -(-n // group)


def _weight(seed, k, count, m, n, group, asym):
    """Codes and grid as a 4-bit quantiser leaves them for Gaussian weights
    of standard deviation 0.02: the group's largest weight on the grid's edge."""
    g = _gen(seed, k)
    codes = torch.empty((count, m, n), dtype=torch.int8, device="cuda")
    ng = _groups(n, group)
    scale = 0.02 / 2.6 * torch.exp(0.15 * torch.randn((count, m, ng), generator=g, device="cuda"))
    zero = None
    if asym:
        zero = torch.randint(6, 10, (count, m, ng), generator=g, device="cuda").float()
    rows = max(1, (1 << 26) // n)
    for e in range(count):
        for r in range(0, m, rows):
            t = torch.randn((min(rows, m - r), n), generator=g, device="cuda").mul_(2.6)
            if asym:
                t.add_(7.5)
            codes[e, r:r + rows] = t.round_().clamp_(*((0, 15) if asym else (-8, 7)))
    return codes, scale, zero


def _samples(seed, k, T, n, dtype, heavy):
    """T rows of n channels; heavy: channel scales drawn log-normal(0, 1)."""
    g = _gen(seed, k)
    x = torch.randn((T, n), generator=g, device="cuda")
    if heavy:
        x *= torch.exp(torch.randn(n, generator=g, device="cuda"))
    return x.to(DTYPES[dtype])


def _inputs(case, seed):
    c = case
    if c["op"] in ("linear", "grad"):
        codes, scale, zero = _weight(seed, 1, 1, c["m"], c["n"], c["group"], c["asym"])
        x = _samples(seed, 2, c["T"], c["n"] if c["op"] == "linear" else c["m"], c["dtype"], c["op"] == "linear")
        return dict(x=x, codes=codes[0], scale=scale[0], zero=None if zero is None else zero[0])
    if c["op"] == "moe":
        wi = _weight(seed, 1, c["E"], 2 * c["f"], c["d"], c["group"], c["asym"])
        wo = _weight(seed, 2, c["E"], c["d"], c["f"], c["group"], c["asym"])
        x = _samples(seed, 3, c["T"], c["d"], c["dtype"], False)
        r = torch.randn((c["E"], c["d"]), generator=_gen(seed, 4), device="cuda") / c["d"] ** 0.5
        return dict(x=x, router=r.to(DTYPES[c["dtype"]]), wi=wi, wo=wo)
    g = _gen(seed, 5)
    x = torch.randn((c["T"], c["d"]), generator=g, device="cuda")
    x = x * torch.exp(0.5 * torch.randn(c["d"], generator=g, device="cuda")) + \
        0.5 * torch.randn((c["T"], 1), generator=g, device="cuda")
    return dict(x=x.to(DTYPES[c["dtype"]]),
                dy=torch.randn((c["T"], c["d"]), generator=g, device="cuda").to(DTYPES[c["dtype"]]),
                gamma=1.0 + 0.1 * torch.randn(c["d"], generator=g, device="cuda"),
                beta=0.1 * torch.randn(c["d"], generator=g, device="cuda"))


EPS = 1e-5


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    kb = _kb()
    dt = DTYPES[case["dtype"]]

    def pack(codes, scale, zero):
        qmin, qmax = (0, 15) if case["asym"] else (-8, 7)
        return kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=case["group"])

    # what a serving or tuning loop keeps: the packed weights, the output and the workspace
    if case["op"] in ("linear", "grad"):
        s["w"] = pack(s.pop("codes"), s.pop("scale"), s.pop("zero"))
        grad = case["op"] == "grad"
        s["out"] = torch.empty((case["T"], case["n"] if grad else case["m"]), dtype=dt, device="cuda")
        s["ws"] = kb.linear_workspace(s["w"], case["T"], dt, grad=grad)
    elif case["op"] == "moe":
        s["wi"], s["wo"] = pack(*s["wi"]), pack(*s["wo"])
        s["out"] = torch.empty((case["T"], case["d"]), dtype=dt, device="cuda")
        s["ws"] = kb.moe_workspace(s["wi"], s["wo"], case["T"], case["k"], dt)
    else:
        s["ws"] = kb.layernorm_grad_workspace(case["T"], case["d"])
    return s


# ---------------------------------------------------------------- one pass

def _value(codes, scale, zero, group):
    """V = s (c - z), fp32."""
    n = codes.shape[-1]
    j = torch.arange(n, device=codes.device) // (group if group else n)
    v = codes.float()
    if zero is not None:
        v = v - zero[..., j]
    return v * scale[..., j]


def _silu(a):
    return a / (1.0 + torch.exp(-a))


def _plain_moe(s, c):
    x = s["x"].float()
    T, E, k = c["T"], c["E"], c["k"]
    logits = x @ s["router"].float().T
    p = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    q, ids = torch.sort(p, dim=1, descending=True, stable=True)
    q, ids = q[:, :k], ids[:, :k]
    q = q / q.sum(dim=1, keepdim=True)
    f = c["f"]

    def at(w, e):
        return _value(w[0][e], w[1][e], None if w[2] is None else w[2][e], c["group"])

    if T * k < E:      # fewer picks than experts: only theirs
        e = ids.reshape(-1)
        xs = x.repeat_interleave(k, dim=0)
        gu = (at(s["wi"], e) @ xs[:, :, None])[:, :, 0]
        h = _silu(gu[:, :f]) * gu[:, f:]
        o = (at(s["wo"], e) @ h[:, :, None])[:, :, 0]
        return (o.reshape(T, k, -1) * q[:, :, None]).sum(dim=1)
    y = torch.zeros_like(x)
    for e in range(E):
        gu = x @ at(s["wi"], e).T
        h = _silu(gu[:, :f]) * gu[:, f:]
        w = (q * (ids == e)).sum(dim=1, keepdim=True)
        y = y + w * (h @ at(s["wo"], e).T)
    return y


def _plain_norm(s):
    x, dy = s["x"].float(), s["dy"].float()
    mu = x.mean(dim=1, keepdim=True)
    xc = x - mu
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1, keepdim=True) + EPS)
    xh = xc * rstd
    y = xh * s["gamma"] + s["beta"]
    a = dy * s["gamma"]
    dx = rstd * (a - a.mean(dim=1, keepdim=True) - xh * (a * xh).mean(dim=1, keepdim=True))
    return dict(y=y.to(s["x"].dtype), dx=dx.to(s["x"].dtype), dgamma=(dy * xh).sum(dim=0), dbeta=dy.sum(dim=0))


def run(state):
    s, c = state, state["case"]
    if own:
        kb = _kb()
        if c["op"] == "linear":
            return kb.bakron_linear(s["x"], s["w"], out=s["out"], workspace=s["ws"])
        if c["op"] == "grad":
            return kb.bakron_linear_grad(s["x"], s["w"], out=s["out"], workspace=s["ws"])
        if c["op"] == "moe":
            return kb.bakron_moe(s["x"], s["router"], s["wi"], s["wo"], c["k"], renormalize=True, out=s["out"],
                                 workspace=s["ws"])
        y, mean, rstd = kb.bakron_layernorm(s["x"], s["gamma"], s["beta"], EPS)
        dx, dgamma, dbeta = kb.bakron_layernorm_grad(s["dy"], s["x"], s["gamma"], mean, rstd, workspace=s["ws"])
        return dict(y=y, dx=dx, dgamma=dgamma, dbeta=dbeta)
    if c["op"] == "linear":
        return (s["x"].float() @ _value(s["codes"], s["scale"], s["zero"], c["group"]).T).to(s["x"].dtype)
    if c["op"] == "grad":
        return (s["x"].float() @ _value(s["codes"], s["scale"], s["zero"], c["group"])).to(s["x"].dtype)
    if c["op"] == "moe":
        return _plain_moe(s, c).to(s["x"].dtype)
    return _plain_norm(s)


def work(case):
    c, e = case, SIZE[case["dtype"]]

    def weight(m, n):   # 4-bit codes, one fp32 scale a group, one byte of zero point where the grid has one
        ng = _groups(n, c["group"])
        return m * n / 2 + m * ng * (5 if c["asym"] else 4)

    if c["op"] in ("linear", "grad"):
        T, m, n = c["T"], c["m"], c["n"]
        return {"bytes": weight(m, n) + e * T * (m + n), "flops": 2 * T * m * n}
    if c["op"] == "moe":
        T, E, k, d, f = c["T"], c["E"], c["k"], c["d"], c["f"]
        distinct = E * (1.0 - (1.0 - k / E) ** T)   # experts that T picks of k of E reach, on average
        return {"bytes": distinct * (weight(2 * f, d) + weight(d, f)) + e * (E * d + 2 * T * d),
                "flops": 2 * T * E * d + 6 * T * k * d * f}
    T, d = c["T"], c["d"]
    return {"bytes": e * T * d * 5 + 16 * d + 8 * T, "flops": 20 * T * d}


# ---------------------------------------------------------------- fp64

def _exact_matrix(codes, scale, zero, group, r0, r1):
    c = codes[r0:r1].double()
    out = torch.empty_like(c)
    n = c.shape[1]
    g = group if group else n
    for k in range(scale.shape[1]):
        sl = slice(k * g, min(n, (k + 1) * g))
        z = 0.0 if zero is None else zero[r0:r1, k:k + 1].double()
        out[:, sl] = (c[:, sl] - z) * scale[r0:r1, k:k + 1].double()
    return out


def _exact_product(x, w, group, transposed=False):
    codes, scale, zero = w
    m = codes.shape[0]
    step = max(1, (1 << 26) // codes.shape[1])
    if transposed:
        out = torch.zeros((x.shape[0], codes.shape[1]), dtype=torch.float64, device=x.device)
        for r in range(0, m, step):
            out += torch.matmul(x[:, r:r + step], _exact_matrix(codes, scale, zero, group, r, min(m, r + step)))
        return out
    return torch.cat([torch.matmul(x, _exact_matrix(codes, scale, zero, group, r, min(m, r + step)).t())
                      for r in range(0, m, step)], dim=1)


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    x = s["x"].double()
    if c["op"] in ("linear", "grad"):
        return _exact_product(x, (s["codes"], s["scale"], s["zero"]), c["group"], c["op"] == "grad")
    if c["op"] == "moe":
        logits = torch.matmul(x, s["router"].double().t())
        y = torch.zeros_like(x)
        of = [(t, e, w) for t in range(c["T"]) for e, w in _picks(logits[t].tolist(), c["k"])]
        for e in sorted({e for _, e, _ in of}):
            rows = [(t, w) for t, e2, w in of if e2 == e]
            xt = x[[t for t, _ in rows]]
            wi = [None if p is None else p[e] for p in s["wi"]]
            wo = [None if p is None else p[e] for p in s["wo"]]
            gu = _exact_product(xt, wi, c["group"])
            gate, up = gu[:, :c["f"]], gu[:, c["f"]:]
            o = _exact_product(gate * torch.sigmoid(gate) * up, wo, c["group"])
            for i, (t, w) in enumerate(rows):
                y[t] += w * o[i]
        return y
    dy, gamma, beta = s["dy"].double(), s["gamma"].double(), s["beta"].double()
    d = c["d"]
    mu = x.sum(1) / d
    var = (x * x).sum(1) / d - mu * mu
    r = (var + EPS).rsqrt()
    xh = (x - mu[:, None]) * r[:, None]
    dgamma = (dy * xh).sum(0)
    g = dy * gamma
    dx = (d * g - g.sum(1)[:, None] - xh * (g * xh).sum(1)[:, None]) * (r / d)[:, None]
    return dict(y=xh * gamma + beta, dx=dx, dgamma=dgamma, dbeta=dy.sum(0))


def _picks(logits, k):
    """The k experts of one token (ties to the lowest index) with weights that sum to 1."""
    import math
    best = sorted(range(len(logits)), key=lambda e: (-logits[e], e))[:k]
    top = logits[best[0]]
    w = [math.exp(logits[e] - top) for e in best]
    return [(e, v / sum(w)) for e, v in zip(best, w)]
