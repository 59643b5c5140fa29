"""Plain 64-bit forms of the quantised layers' operators and the error bounds
their tests use.

Rounding bounds (u = 2^-24, fp32 unit roundoff).  An output is a sum formed
in fp32 and rounded once to its type: the last rounding is at most half an
ulp, HALF_ULP[dtype] relative.  The sum itself: with every addition or
multiplication relative error at most 2 u (the tensor cores may cut off
instead of rounding), a sum of terms t_i that any single term reaches through
at most D additions is within D 2 u sum |t_i| of the exact one (first order).
"""

import torch

U = 2.0 ** -24
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def bound(abs_sum, depth, dtype, value):
    """Largest accepted error: `depth` additions in fp32 over terms whose
    magnitudes sum to abs_sum, then one rounding of `value` to dtype."""
    err = 2.0 * U * depth * abs_sum
    return err + HALF_ULP[dtype] * (value.abs() + err) + TINY[dtype]


def product_depth(n, terms=3):
    """Additions a term of a length-n product passes: the 128-column partial
    sum on the tensor cores (16 columns an instruction, up to `terms` terms of
    each activation), then one addition per 128 columns at worst, one
    multiplication by the scale and a few joins."""
    return 128 * terms / 16 + 16 + (n + 127) // 32 + 32


def value(codes, scale, zero, group):
    """V = s (c - z), fp64, any leading dimensions."""
    n = codes.shape[-1]
    g = group if group and group < n else n
    j = torch.arange(n, device=codes.device) // g
    v = codes.double()
    s = scale.double()
    if s.dim() < codes.dim():
        s = s.unsqueeze(-1)
    if zero is not None:
        z = zero.double()
        v = v - (z if z.dim() == codes.dim() else z.unsqueeze(-1))[..., j]
    return v * s[..., j]


def random_weight(shape, group, asym, seed, bits=4, device="cuda"):
    """Random codes and grid: (codes, scale, zero, qmin, qmax)."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    n = shape[-1]
    ng = 1 if not group or group >= n else -(-n // group)
    qmin, qmax = (0, (1 << bits) - 1) if asym else (-(1 << (bits - 1)), (1 << (bits - 1)) - 1)
    codes = torch.randint(qmin, qmax + 1, shape, generator=g, dtype=torch.int8)
    scale = torch.exp(torch.randn(shape[:-1] + (ng,), generator=g)) * 0.01
    zero = torch.randint(qmin, qmax + 1, shape[:-1] + (ng,), generator=g).float() if asym else None
    put = lambda t: None if t is None else t.to(device)
    return put(codes), put(scale), put(zero), qmin, qmax
