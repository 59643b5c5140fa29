"""Cases for the operators of a block's feed-forward part over quantised
weights: the product with bias, activation and residual in its epilogue, the
activation alone with its gradient, tokens sorted by expert and back, and the
experts' products over sorted tokens in both directions.

``run`` is one pass: with ``own`` false from elementary torch operations in
fp32, rounded once at the end; with ``own`` true through the framework's entry
points.  ``exact`` is the same pass from the definition in fp64.
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def listed():
    return [
        # one new token through a small layer with bias and activation: latency is all that counts
        dict(name="linear_act_1_1024x1024", op="linear_act", T=1, m=1024, n=1024, group=128, asym=False, dtype="bf16",
             act="silu", bias=True, residual=False, pre=False),
        # a batch of sequences decoding through an MLP's first layer
        dict(name="linear_act_48_14336x4096", op="linear_act", T=48, m=14336, n=4096, group=64, asym=True,
             dtype="fp16", act="gelu_tanh", bias=True, residual=False, pre=False),
        # a tuning batch: the activation's input is kept for the backward pass, the stream's residual is added
        dict(name="linear_act_2048_8192x8192", op="linear_act", T=2048, m=8192, n=8192, group=128, asym=False,
             dtype="bf16", act="silu", bias=True, residual=True, pre=True),
        # the activation of a few odd rows forward and back, with the bias's gradient, in the solver's own type
        dict(name="act_37_1111_fp32", op="act", T=37, m=1111, dtype="fp32", act="gelu", gated=False, bias=True),
        # a tuning batch's gated activation, forward and back
        dict(name="act_2048_14336_gated", op="act", T=2048, m=14336, dtype="bf16", act="silu", gated=True, bias=False),
        # a few sequences decoding: sorted by expert and laid out, many small experts
        dict(name="sort_16_e32k4_1024", op="sort", T=16, E=32, k=4, d=1024, dtype="bf16", index="int64", pad=0.0),
        # a training batch with some padding
        dict(name="sort_8192_e64k6_4096", op="sort", T=8192, E=64, k=6, d=4096, dtype="bf16", index="int64", pad=0.05),
        # back again with weights, forward and gradients: a calibration batch in fp32, odd rows
        dict(name="combine_333_e8k2_1111_fp32", op="combine", T=333, E=8, k=2, d=1111, dtype="fp32", pad=0.0),
        # the same for a training batch
        dict(name="combine_8192_e8k2_4096", op="combine", T=8192, E=8, k=2, d=4096, dtype="bf16", pad=0.0),
        # a batch of sequences decoding through many small experts, a handful of tokens each
        dict(name="experts_64_e32k4_1408x1024", op="experts", T=64, E=32, k=4, m=1408, n=1024, group=64, asym=False,
             dtype="bf16", pad=0.0, grad=False),
        # a prompt through the wide experts' gate and up projections
        dict(name="experts_2048_e8k2_28672x4096", op="experts", T=2048, E=8, k=2, m=28672, n=4096, group=128,
             asym=False, dtype="bf16", pad=0.0, grad=False),
        # a tuning batch's gradient through the experts' down projections
        dict(name="experts_grad_2048_e8k2_4096x14336", op="experts", T=2048, E=8, k=2, m=4096, n=14336, group=128,
             asym=True, dtype="bf16", pad=0.0, grad=True),
    ]


def _log(rng, lo, hi):
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.4:   # real layers are mostly multiples of 64, some sizes are odd
        return max(lo, min(hi, v))
    return max(lo, min(hi, max(64, v // 64 * 64) if hi >= 64 and v >= 64 else v))


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def draw(rng):
    op = rng.choice(["linear_act", "linear_act", "act", "sort", "combine", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    weight = dict(group=rng.choice([0, 32, 64, 96, 128, 128, 256]), asym=rng.random() < 0.5)
    pad = rng.choice([0.0, 0.0, 0.05, 0.3])
    E = rng.choice([4, 8, 16, 32, 60, 64, 128])
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    while True:
        if op == "linear_act":
            c = dict(op=op, T=_log(rng, 1, 2048), m=_log(rng, 100, 14336), n=_log(rng, 100, 14336), dtype=dtype,
                     act=rng.choice(ACTS), bias=rng.random() < 0.7, residual=rng.random() < 0.5,
                     pre=rng.random() < 0.4, **weight)
            if c["T"] * c["m"] * c["n"] > 2048 * 8192 * 8192 // (4 if dtype == "fp32" else 1):
                continue
        elif op == "act":
            c = dict(op=op, T=_log(rng, 1, 8192), m=_log(rng, 64, 14336), dtype=dtype, act=rng.choice(ACTS[1:]),
                     gated=rng.random() < 0.5, bias=rng.random() < 0.4)
            if c["T"] * c["m"] > 2048 * 14336:
                continue
        elif op in ("sort", "combine"):
            c = dict(op=op, T=_log(rng, 1, 8192), E=E, k=k, d=_log(rng, 64, 8192), dtype=dtype, pad=pad)
            if op == "sort":
                c["index"] = rng.choice(["int32", "int64"])
            if c["T"] * (c["k"] + 1) * c["d"] * SIZE[dtype] > 8192 * 7 * 4096 * 2:
                continue
        else:
            c = dict(op=op, T=_log(rng, 1, 2048), E=E, k=k, m=_log(rng, 100, 14336), n=_log(rng, 100, 14336),
                     dtype=dtype, pad=pad, grad=rng.random() < 0.5, **weight)
            if c["T"] * k * c["m"] * c["n"] > 4096 * 28672 * 4096 // (4 if dtype == "fp32" else 1):
                continue
            if E * c["m"] * c["n"] > 8 * 28672 * 4096:
                continue
        return c


# ---------------------------------------------------------------- inputs

def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + k)


def _groups(n, group):
    return 1 if not group or group >= n else -(-n // group)


def _weight(seed, count, m, n, group, asym):
    """Codes and grid as a 4-bit quantiser leaves them for Gaussian weights
    of standard deviation 0.02: the group's largest weight on the grid's edge."""
    g = _gen(seed, 1)
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


def _randn(seed, k, shape, dtype, spread=1.0):
    return (spread * torch.randn(shape, generator=_gen(seed, k), device="cuda")).to(DTYPES[dtype])


def _choices(seed, T, E, k, pad):
    """k distinct experts per token, some more popular than others, and their
    weights (softmax of the chosen logits); a padding token has chosen -1."""
    g = _gen(seed, 7)
    logits = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    top, choice = torch.topk(logits, k, dim=1)
    if pad:
        choice[torch.rand(T, generator=g, device="cuda") < pad] = -1
    return choice, torch.softmax(top, dim=1)


def _places(choice, E):
    """Offsets of the experts' rows and the row of every choice (-1: none):
    the choices ordered by expert, within an expert as they come."""
    flat = choice.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(len(order), device=order.device)
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device=key.device))
    place = torch.where(key < E, row, torch.full_like(row, -1))
    return offsets.int(), place.int().reshape(choice.shape)


def _inputs(case, seed):
    c = case
    dt = c["dtype"]
    if c["op"] == "linear_act":
        codes, scale, zero = _weight(seed, 1, c["m"], c["n"], c["group"], c["asym"])
        return dict(x=_randn(seed, 2, (c["T"], c["n"]), dt), codes=codes, scale=scale, zero=zero,
                    bias=_randn(seed, 3, (c["m"],), "fp32", 0.3) if c["bias"] else None,
                    residual=_randn(seed, 4, (c["T"], c["m"]), dt) if c["residual"] else None)
    if c["op"] == "act":
        return dict(z=_randn(seed, 2, (c["T"], c["m"] * (2 if c["gated"] else 1)), dt, 1.5),
                    dy=_randn(seed, 3, (c["T"], c["m"]), dt))
    choice, weight = _choices(seed, c["T"], c["E"], c["k"], c["pad"])
    if c["op"] == "sort":
        return dict(choice=choice.to(getattr(torch, c["index"])), x=_randn(seed, 2, (c["T"], c["d"]), dt))
    offsets, place = _places(choice, c["E"])
    rows = c["T"] * c["k"]
    if c["op"] == "combine":
        return dict(place=place, weight=weight, rows=_randn(seed, 2, (rows, c["d"]), dt),
                    dy=_randn(seed, 3, (c["T"], c["d"]), dt))
    codes, scale, zero = _weight(seed, c["E"], c["m"], c["n"], c["group"], c["asym"])
    return dict(x=_randn(seed, 2, (rows, c["m"] if c["grad"] else c["n"]), dt), offsets=offsets, codes=codes,
                scale=scale, zero=zero)


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = c
    dt = DTYPES[c["dtype"]]
    # what a serving or tuning loop keeps: outputs (rows that no token has stay zero), packed weights, workspaces
    if c["op"] == "linear_act":
        s["out"] = torch.zeros((c["T"], c["m"]), dtype=dt, device="cuda")
        s["pre"] = torch.zeros_like(s["out"]) if c["pre"] else None
    elif c["op"] == "act":
        s["y"], s["dz"] = torch.zeros_like(s["dy"]), torch.zeros_like(s["z"])
    elif c["op"] == "sort":
        s["out"] = torch.zeros((c["T"] * c["k"], c["d"]), dtype=dt, device="cuda")
        s["offsets"] = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
        s["place"] = torch.zeros((c["T"], c["k"]), dtype=torch.int32, device="cuda")
    elif c["op"] == "combine":
        s["y"], s["drows"] = torch.zeros_like(s["dy"]), torch.zeros_like(s["rows"])
        s["dweight"] = torch.zeros_like(s["weight"])
    else:
        s["out"] = torch.zeros((c["T"] * c["k"], c["n"] if c["grad"] else c["m"]), dtype=dt, device="cuda")
    if not own:
        return s
    kb = _kb()
    if "codes" in s:
        codes, scale, zero = s.pop("codes"), s.pop("scale"), s.pop("zero")
        if c["op"] == "linear_act":
            codes, scale, zero = codes[0], scale[0], None if zero is None else zero[0]
        qmin, qmax = (0, 15) if c["asym"] else (-8, 7)
        s["w"] = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=c["group"])
    if c["op"] == "linear_act":
        s["ws"] = kb.linear_workspace(s["w"], c["T"], dt)
    elif c["op"] == "act":
        s["ws"] = kb.act_grad_workspace(c["T"], s["z"].shape[1]) if c["bias"] else None
    elif c["op"] == "experts":
        s["ws"] = kb.experts_workspace(s["w"], c["T"] * c["k"], dt, grad=c["grad"])
    return s


# ---------------------------------------------------------------- one pass

def _value(codes, scale, zero, group):
    """V = s (c - z), fp32."""
    n = codes.shape[-1]
    j = torch.arange(n, device=codes.device) // (group if group else n)
    v = codes.float()
    if zero is not None:
        v -= zero[..., j]
    return v.mul_(scale[..., j])


SQRT_HALF = math.sqrt(0.5)
GELU_TANH = math.sqrt(2.0 / math.pi)


def _act(z, act):
    """(a(z), a'(z)) of an fp32 tensor."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":   # the tail by erfc, which does not cancel
        p = 0.5 * torch.special.erfc(-SQRT_HALF * z)
        return z * p, p + z * torch.exp(-0.5 * z * z) * (0.5 * GELU_TANH)
    # 0.5 (1 + tanh u) = 1 / (1 + exp(-2 u))
    s = 1.0 / (1.0 + torch.exp(-2.0 * GELU_TANH * (z + 0.044715 * z * z * z)))
    return z * s, s + z * s * (1.0 - s) * 2.0 * GELU_TANH * (1.0 + 3 * 0.044715 * z * z)


def _plain_act(s, c):
    z, dy = s["z"].float(), s["dy"].float()
    if c["gated"]:
        g, u = z[:, :c["m"]], z[:, c["m"]:]
        a, da = _act(g, c["act"])
        y, dz = a * u, torch.cat([dy * u * da, dy * a], dim=1)
    else:
        a, da = _act(z, c["act"])
        y, dz = a, dy * da
    out = dict(y=y.to(s["z"].dtype), dz=dz.to(s["z"].dtype))
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


def _plain_combine(s):
    there = (s["place"] >= 0)[..., None]
    at = s["place"].clamp(min=0).long()
    rows = s["rows"].float()[at] * there                        # (T, k, d)
    y = (rows * s["weight"][..., None]).sum(dim=1)
    dy = s["dy"].float()[:, None, :]
    s["drows"][at[there[..., 0]]] = (dy * s["weight"][..., None])[there[..., 0]].to(s["rows"].dtype)
    return dict(y=y.to(s["rows"].dtype), drows=s["drows"], dweight=(rows * dy).sum(dim=2))


def _plain_experts(s, c):
    bounds = s["offsets"].tolist()
    for e in range(c["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        v = _value(s["codes"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e], c["group"])
        s["out"][lo:hi] = (s["x"][lo:hi].float() @ (v if c["grad"] else v.T)).to(s["x"].dtype)
    return s["out"]


def run(state):
    s, c = state, state["case"]
    if own:
        kb = _kb()
        if c["op"] == "linear_act":
            y, pre = kb.bakron_linear_act(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                          want_pre=c["pre"], out=s["out"], pre=s["pre"], workspace=s["ws"])
            return dict(y=y, pre=pre) if c["pre"] else dict(y=y)
        if c["op"] == "act":
            y = kb.bakron_act(s["z"], c["act"], gated=c["gated"], out=s["y"])
            dz, dbias = kb.bakron_act_grad(s["dy"], s["z"], c["act"], gated=c["gated"], want_bias_grad=c["bias"],
                                           out=s["dz"], workspace=s["ws"])
            return dict(y=y, dz=dz, dbias=dbias) if c["bias"] else dict(y=y, dz=dz)
        if c["op"] == "sort":
            offsets, place = kb.bakron_sort_tokens(s["choice"], c["E"], out=(s["offsets"], s["place"]))
            return dict(offsets=offsets, place=place, rows=kb.bakron_dispatch(s["x"], place, out=s["out"]))
        if c["op"] == "combine":
            y = kb.bakron_combine(s["rows"], s["place"], s["weight"], out=s["y"])
            drows, dweight = kb.bakron_combine_grad(s["dy"], s["rows"], s["place"], s["weight"],
                                                    out=(s["drows"], s["dweight"]))
            return dict(y=y, drows=drows, dweight=dweight)
        product = kb.bakron_experts_grad if c["grad"] else kb.bakron_experts
        return product(s["x"], s["w"], s["offsets"], out=s["out"], workspace=s["ws"])
    if c["op"] == "linear_act":
        v = _value(s["codes"][0], s["scale"][0], None if s["zero"] is None else s["zero"][0], c["group"])
        z = s["x"].float() @ v.T
        if c["bias"]:
            z = z + s["bias"]
        y = _act(z, c["act"])[0]
        if c["residual"]:
            y = y + s["residual"].float()
        out = dict(y=y.to(s["x"].dtype))
        if c["pre"]:
            out["pre"] = z.to(s["x"].dtype)
        return out
    if c["op"] == "act":
        return _plain_act(s, c)
    if c["op"] == "sort":
        offsets, place = _places(s["choice"], c["E"])
        there = place >= 0
        s["out"][place[there].long()] = s["x"][:, None, :].expand(-1, c["k"], -1)[there]
        return dict(offsets=offsets, place=place, rows=s["out"])
    if c["op"] == "combine":
        return _plain_combine(s)
    return _plain_experts(s, c)


def work(case):
    c, e = case, SIZE[case["dtype"]]

    def weight(m, n):   # 4-bit codes, one fp32 scale a group, one byte of zero point where the grid has one
        ng = _groups(n, c["group"])
        return m * n / 2 + m * ng * (5 if c["asym"] else 4)

    if c["op"] == "linear_act":
        T, m, n = c["T"], c["m"], c["n"]
        return {"bytes": weight(m, n) + e * T * (n + m * (1 + c["residual"] + c["pre"])) + 4 * m * c["bias"],
                "flops": 2 * T * m * n}
    if c["op"] == "act":
        T, m = c["T"], c["m"]
        z = 2 * m if c["gated"] else m
        return {"bytes": e * T * (2 * z + 2 * m) + 4 * z * c["bias"], "flops": 20 * T * m}
    T, k = c["T"], c["k"]
    rows = T * k * (1.0 - c["pad"])
    if c["op"] == "sort":
        index = 4 if c["index"] == "int32" else 8
        return {"bytes": T * k * (index + 4) + 4 * (c["E"] + 1) + e * c["d"] * (T + rows), "flops": T * k}
    if c["op"] == "combine":
        return {"bytes": e * c["d"] * (2 * T + 2 * rows) + 12 * T * k, "flops": 5 * rows * c["d"]}
    # experts that any token reaches, on average
    distinct = c["E"] * (1.0 - (1.0 - k / c["E"]) ** (T * (1.0 - c["pad"])))
    return {"bytes": distinct * weight(c["m"], c["n"]) + e * rows * (c["m"] + c["n"]) + 4 * (c["E"] + 1),
            "flops": 2 * rows * c["m"] * c["n"]}


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


def _exact_product(x, w, group, transposed):
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


def _exact_gain(z, act):
    """(a(z) / z, a'(z)) in fp64."""
    if act == "none":
        return torch.ones_like(z), torch.ones_like(z)
    if act == "relu":
        on = (z > 0).double()
        return on, on
    if act == "silu":
        p = torch.sigmoid(z)
        return p, p * (1 + z * torch.sigmoid(-z))
    if act == "gelu":
        p = torch.special.erfc(-z / math.sqrt(2.0)) / 2
        return p, p + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    u = c * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(2 * u)
    return p, p + z * 2 * p * torch.sigmoid(-2 * u) * c * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "linear_act":
        z = _exact_product(s["x"].double(), (s["codes"][0], s["scale"][0], None if s["zero"] is None else s["zero"][0]),
                           c["group"], False)
        if c["bias"]:
            z += s["bias"].double()
        y = z * _exact_gain(z, c["act"])[0]
        if c["residual"]:
            y += s["residual"].double()
        return dict(y=y, pre=z) if c["pre"] else dict(y=y)
    if c["op"] == "act":
        z, dy = s["z"].double(), s["dy"].double()
        g = z[:, :c["m"]]
        gain, slope = _exact_gain(g, c["act"])
        if c["gated"]:
            u = z[:, c["m"]:]
            y, dz = g * gain * u, torch.cat([dy * u * slope, dy * g * gain], dim=1)
        else:
            y, dz = g * gain, dy * slope
        return dict(y=y, dz=dz, dbias=dz.sum(0)) if c["bias"] else dict(y=y, dz=dz)
    if c["op"] == "sort":
        # the row of a choice: all choices of lower experts, then the earlier ones of its own
        flat = s["choice"].reshape(-1).long()
        hits = flat[:, None] == torch.arange(c["E"], device=flat.device)[None, :]
        counts = hits.sum(0)
        first = torch.cumsum(counts, 0) - counts
        before = torch.cumsum(hits.int(), 0) - hits.int()
        live = hits.any(1)
        place = torch.where(live, ((before + first) * hits).sum(1), torch.full_like(flat, -1)).int()
        offsets = torch.cat([first, counts.sum()[None]]).int()
        rows = torch.zeros((c["T"] * c["k"], c["d"]), dtype=torch.float64, device="cuda")
        token = torch.arange(len(flat), device="cuda") // c["k"]
        rows[place[live].long()] = s["x"].double()[token[live]]
        return dict(offsets=offsets, place=place.reshape(c["T"], c["k"]), rows=rows)
    if c["op"] == "combine":
        rows, dy, weight = s["rows"].double(), s["dy"].double(), s["weight"].double()
        y, drows, dweight = torch.zeros_like(dy), torch.zeros_like(rows), torch.zeros_like(weight)
        for j in range(c["k"]):
            t = torch.nonzero(s["place"][:, j] >= 0)[:, 0]
            r = s["place"][t, j].long()
            y[t] += weight[t, j, None] * rows[r]
            drows[r] = weight[t, j, None] * dy[t]
            dweight[t, j] = (rows[r] * dy[t]).sum(1)
        return dict(y=y, drows=drows, dweight=dweight)
    out = torch.zeros((c["T"] * c["k"], c["n"] if c["grad"] else c["m"]), dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist()
    for e in range(c["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            w = (s["codes"][e], s["scale"][e], None if s["zero"] is None else s["zero"][e])
            out[lo:hi] = _exact_product(s["x"][lo:hi].double(), w, c["group"], c["grad"])
    return out
