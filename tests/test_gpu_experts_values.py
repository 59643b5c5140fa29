"""The experts' products where a term of an fp32 operand, a plane's row or the scales' common factor
would be wrong without showing in sums of many random terms."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, bound, product_depth, random_weight, value

pytestmark = pytest.mark.gpu


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _offsets(counts, first):
    return torch.tensor([first + sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_one_expert_is_the_linear_layer(dtype, grad):
    """All rows in one expert, at a size where both take whole columns: the same bits."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((1, 2560, 2560), 128, False, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, group=128)
    x = _randn((2000, 2560), dtype, 4)
    offsets = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    a = (kb.bakron_experts_grad if grad else kb.bakron_experts)(x, w, offsets)
    b = (kb.bakron_linear_grad if grad else kb.bakron_linear)(x, w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("counts,first,m,n,group", [
    ([5, 0, 70, 1], 3, 130, 260, 32), ([40, 90], 1, 300, 515, 96), ([2, 150, 33], 7, 70, 256, 64), ([64, 65], 0, 257, 640, 128),
    ([9] * 20, 2, 40, 130, 0)])
def test_all_bits_of_fp32(counts, first, m, n, group, grad):
    """One non-zero per row, with all 24 bits in use, and experts that begin at rows other than 0:
    every result is a single product, so that each term of its operands counts.

    In units of u = 2^-24 of the value.  Forward: the first term's product is exact (8 and 5 bits), the
    sum of the two small ones is off by at most 2 u 2^-7, joining them 2 u, the scale's product u; zeros
    are added exactly.  Backward: the weight's own product u, the three left out u, the five small
    ones' sums below 5 (2 u) 2^-7, joining 2 u.  Below 4.2 u either way; without the last of three
    terms a value is off by up to 2^-17 = 128 u, half of that on average."""
    kb = _kb()
    E, R = len(counts), first + sum(counts) + 2
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), group, True, m + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    offsets = _offsets(counts, first)
    K, N = (m, n) if grad else (n, m)
    g = torch.Generator().manual_seed(R)
    at = torch.randint(0, K, (R,), generator=g).cuda()
    bits = torch.randint(1 << 23, 1 << 24, (R,), generator=g).float().cuda()     # odd ones too: 24 bits
    x = torch.zeros((R, K), device="cuda")
    x[torch.arange(R, device="cuda"), at] = bits * torch.where(at % 2 == 0, 2.0 ** -23, -2.0 ** -20)
    out = torch.full((R, N), 7.0, device="cuda")
    (kb.bakron_experts_grad if grad else kb.bakron_experts)(x, w, offsets, out=out)
    kb.bakron_async_status()
    o = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(o, o[1:])):
        ref = x[lo:hi].double() @ (V[e] if grad else V[e].T)
        assert ((out[lo:hi].double() - ref).abs() <= 4.2 * 2.0 ** -24 * ref.abs()).all(), "expert %d" % e
    assert (out[:first] == 7.0).all() and (out[o[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("steps", [10, 20, 30])
def test_gradient_of_experts_of_different_scales(steps, dtype):
    """Three experts, each 2^-steps of the one before it for half of them.  The scales of all share a
    power of two; in fp16, weights below 2^-25 of the largest scale lose bits, at most half of the
    smallest fp16 number as it is then: 2^-36 of the largest scale."""
    kb = _kb()
    E, m, n = 3, 200, 260
    codes, _, zero, qmin, qmax = random_weight((E, m, n), 64, True, steps)
    scale = 0.01 * (1 + torch.rand((E, m, 5), generator=torch.Generator().manual_seed(steps)))
    scale = (scale * torch.tensor([1.0, 2.0 ** -steps, 2.0 ** -(steps // 2)])[:, None, None]).cuda()
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    V = value(codes, scale, zero, 64)
    counts = [30, 41, 50]
    offsets = _offsets(counts, 0)
    dy = _randn((sum(counts), m), dtype, 2) * 4096          # so that the smallest results are normal numbers
    dx = kb.bakron_experts_grad(dy, w, offsets)
    o = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(o, o[1:])):
        d = dy[lo:hi].double()
        ref, mag = d @ V[e], d.abs() @ V[e].abs()
        tol = bound(mag, product_depth(m, terms=6), dtype, ref)
        if dtype != torch.float32:
            tol = tol + HALF_ULP[dtype] * mag
        if dtype == torch.float16:
            tol = tol + 2.0 ** -36 * scale.max().item() * d.abs().sum(1, keepdim=True)
        assert ((dx[lo:hi].double() - ref).abs() <= tol).all(), "expert %d" % e
