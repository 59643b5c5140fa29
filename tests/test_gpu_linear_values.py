"""The quantised layers over the whole range of their values."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, TINY, U, bound, product_depth, random_weight, value

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _dy(T, m, dtype, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn((T, m), generator=g).to(dtype).cuda()


# Scales over the whole range that bakron_pack takes, with gradients for which the results are finite and
# normal: (log2 of the scales' middle, spread in octaves either way, log2 of dY).
RANGES = {torch.float16: [(13, 1, -13), (20, 2, -22), (-16, 2, 6), (-26, 3, 10), (-4, 8, 0)],
          torch.bfloat16: [(122, 2, -30), (-130, 2, 60), (-60, 10, 20), (40, 5, 0)],
          torch.float32: [(122, 2, -30), (-130, 2, 60), (-60, 10, 20), (40, 5, 0)]}

@pytest.mark.parametrize("dtype,mid,spread,mag", [(d, *r) for d in DTYPES for r in RANGES[d]])
@pytest.mark.parametrize("T,m,n,group,asym", [(33, 150, 300, 0, False), (130, 700, 260, 64, True)])
def test_scales_of_any_size(T, m, n, group, asym, dtype, mid, spread, mag):
    """V is rounded once to dY's type, relative to each weight, whatever the
    scales' size; fp32 weights are not rounded."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m)
    g = torch.Generator(device="cpu").manual_seed(m)
    e = mid + spread * (2 * torch.rand(scale.shape, generator=g, dtype=torch.float64) - 1)
    scale = torch.exp2(e).float().cuda()
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    dy = (_dy(T, m, torch.float32, n) * 2.0 ** mag).to(dtype)
    dx = kb.bakron_linear_grad(dy, w)
    ref = dy.double() @ V
    abs_sum = dy.double().abs() @ V.abs()
    tol = bound(abs_sum, product_depth(m, terms=6), dtype, ref)
    if dtype != torch.float32:
        tol = tol + HALF_ULP[dtype] * abs_sum
    assert torch.isfinite(dx).all()
    worst = ((dx.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "error %.3g times the bound" % worst
