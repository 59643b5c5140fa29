"""Plain 64-bit forms of the activations and of tokens sorted by expert, and the
error bounds of their tests (u = 2^-24, see _layer_helpers).

An activation in fp32.  Its argument's error, relative 2 u at most where the argument is
computed (z^2, its multiple, the sum: 6 u), reaches the result through the exponential: relative
to the result |z q| (1 - s) for z s with s = 1 / (1 + exp(-z q)), and z^2 for gelu's tail
(erfc(x) falls as exp(-x^2), x^2 = z^2 / 2, twice its relative change), nothing where the
result is z itself.  The functions: exp at most 2 + 1.2 |x| units in the last place (the fast
form of 16-bit results), 2 for the other, erfc 4, a division 2, each at most 2 u; a product or
sum u each.  Sixteen of these cover what does not grow with the argument.
"""

import math

import torch

from _layer_helpers import HALF_ULP, TINY, U

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def activation(z, act):
    """(a, a', error of fp32 a, error of fp32 a') of z in fp64, as long as z is finite."""
    zero, one = torch.zeros_like(z), torch.ones_like(z)
    if act == "none":
        return z, one, zero, zero
    if act == "relu":
        on = (z > 0).double()
        return z * on, on, zero, zero
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        density = torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        e = U * (32 + 8 * z * z * (z < 0))
        ed = U * (32 + 8 * z * z)
        return z * p, p + z * density, (z * p).abs() * e, p * e + (z * density).abs() * ed
    if act == "silu":
        q, dq = one, one
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        q, dq = c * (1 + 0.044715 * z * z), c * (1 + 3 * 0.044715 * z * z)
    s, t = torch.sigmoid(z * q), torch.sigmoid(-z * q)
    arg = (z * q).abs().clamp(max=800)
    e = U * (32 + 12 * arg * t)
    # 1 - s is a difference: off by u s and by the error of s
    slope = s + z * s * t * dq
    eslope = s * e + (z * dq * s).abs() * (t * (e + 16 * U) + s * (e + 2 * U))
    return z * s, slope, (z * s).abs() * e, torch.where(s == 0, zero, eslope)


def small(dtype):
    """What results below the normal range may be off by (divisions of huge numbers give 0)."""
    return TINY[dtype] + 2.0 ** -125


def rounded(err, value, dtype):
    """The error bound of an fp32 value of that error, after its rounding to dtype."""
    return err + HALF_ULP[dtype] * (value.abs() + err) + small(dtype)


def check(got, want, err, what=""):
    assert got.shape == want.shape
    assert torch.isfinite(got).all(), what
    worst = ((got.double() - want).abs() / err).max().item() if want.numel() else 0.0
    assert worst <= 1.0, "%s: error %.3g times the bound" % (what, worst)


def places(choice, E):
    """(offsets, place) of choices as lists: by expert, within one as they come."""
    T, k = choice.shape
    flat = choice.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(i)
    place, offsets = [-1] * len(flat), [0]
    for of in rows:
        for n, i in enumerate(of):
            place[i] = offsets[-1] + n
        offsets.append(offsets[-1] + len(of))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(place, dtype=torch.int32).reshape(T, k)


def random_choices(T, k, E, seed, lost=0.1):
    """k experts per token, some twice, some outside the range."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, E, (T, k), generator=g)
    out = torch.rand((T, k), generator=g) < lost
    return torch.where(out, torch.randint(0, 2, (T, k), generator=g) * (E + 3) - 2, c)
