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


def formula(dy, V):
    """sum_i dy_ti V_ij in fp64, term by term, so that infinities and NaN
    meet every weight of their row as written."""
    out = torch.zeros((dy.shape[0], V.shape[1]), dtype=torch.float64, device=dy.device)
    for i in range(dy.shape[1]):
        out += dy[:, i:i + 1].double() * V[i:i + 1]
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym", [
    (9, 100, 300, 0, False), (40, 600, 257, 32, True), (70, 1100, 130, 128, True), (700, 64, 4200, 96, False)])
def test_infinities_and_nan_as_in_the_formula(T, m, n, group, asym, dtype):
    """Scales are powers of two and codes small, so every weight fits in one
    bf16 term: the second and third terms of an fp32 product are exact zeros,
    which an infinite gradient must not meet."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m)
    scale = torch.exp2(torch.round(torch.log2(scale)))
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    dy = _dy(T, m, dtype, n)
    inf = float("inf")
    dy[1, m // 2] = inf
    dy[2, 3] = -inf
    dy[3, 0] = inf
    dy[3, m - 1] = inf
    dy[4, 5] = inf
    dy[4, 6] = -inf
    dy[5, m - 2] = float("nan")
    dy[T - 1, 7] = inf
    dx = kb.bakron_linear_grad(dy, w)
    ref = formula(dy, V)
    assert torch.equal(torch.isnan(dx), torch.isnan(ref))
    assert torch.equal(dx == inf, ref == inf) and torch.equal(dx == -inf, ref == -inf)
    ok = torch.isfinite(ref)
    tol = bound(dy.double().abs().nan_to_num(0, 0, 0) @ V.abs(), product_depth(m, terms=6), dtype, ref)
    assert ((dx.double() - ref).abs()[ok] <= tol[ok]).all()
    kb.bakron_async_status()


def test_a_sum_that_overflows_stays_infinite():
    kb = _kb()
    codes = torch.full((40, 130), 7, dtype=torch.int8, device="cuda")
    w = kb.bakron_pack(codes, torch.ones((40, 1), device="cuda"), -8, 7)
    dy = torch.full((5, 40), 3e38, device="cuda")
    dy[1] = -dy[1]
    dy[2] = 1.0
    dx = kb.bakron_linear_grad(dy, w)
    assert (dx[0] == float("inf")).all() and (dx[1] == float("-inf")).all() and (dx[2] == 280).all()


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


def test_products_of_full_precision():
    """One product per output (m = 1).  With x = hi + mid + lo in rounded bf16
    terms mid is at most 2^-8 and lo at most 2^-17 of the power of two below x, so the
    three products left out are at most 2^-24 (1 + 2^-9) of the whole; the two
    sums' addition rounds once more, 2^-24."""
    kb = _kb()
    g = torch.Generator(device="cpu").manual_seed(4)
    n, T = 4, 4000
    for trial in range(4):
        s = torch.exp2(4 * torch.rand((1, 1), generator=g)).cuda()
        dy = torch.exp2(4 * torch.rand((T, 1), generator=g)).cuda()
        if trial == 0:
            s.fill_(1 + 2.0 ** -7 - 2.0 ** -23)
            dy[:10] = 1 + 2.0 ** -7 - 2.0 ** -23
        codes = torch.ones((1, n), dtype=torch.int8, device="cuda")
        w = kb.bakron_pack(codes, s, -8, 7)
        dx = kb.bakron_linear_grad(dy, w)
        ref = dy.double() * s.double() * torch.ones((1, n), device="cuda").double()
        worst = ((dx.double() - ref).abs() / ref).max().item()
        assert worst <= 2.1 * U, "error %.3g of 2^-24" % (worst / U)


@pytest.mark.parametrize("T,m,n,dtype", [(64, 131072, 130, torch.float16), (300, 65600, 2048, torch.float16),
                                         (1, 100000, 60, torch.float16), (40, 131072, 256, torch.bfloat16),
                                         (600, 9000, 8200, torch.float16), (600, 33000, 8200, torch.bfloat16)])
def test_long_sums(T, m, n, dtype):
    """Sums of one sign over many rows: the tensor core cuts a sum off at
    every addition (at most 2^-23 of it, one per 16 rows), so a chain of them is
    at most 4096 rows long (bf16: 32768), 2^-15 (2^-12); the chains are added with
    roundings of 2^-24."""
    kb = _kb()
    g = torch.Generator(device="cpu").manual_seed(T)
    codes = torch.randint(1, 8, (m, n), generator=g, dtype=torch.int8).cuda()
    w = kb.bakron_pack(codes, torch.full((m, 1), 2.0 ** -6, device="cuda"), -8, 7)     # V is exact
    dy = (0.01 + 0.05 * torch.rand((T, m), generator=g)).to(dtype).cuda()
    dx = kb.bakron_linear_grad(dy, w)
    ref = dy.double() @ (codes.double() * 2.0 ** -6)
    chain = 4096 if dtype == torch.float16 else 32768
    err = (chain / 16 * 2.0 ** -23 + (m / chain + 8) * U) * ref
    tol = err + HALF_ULP[dtype] * (ref + err) + TINY[dtype]
    worst = ((dx.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "error %.3g times the bound" % worst
    assert torch.equal(dx, kb.bakron_linear_grad(dy, w))


def test_experts_hidden_values_keep_sixteen_bits():
    """One token, one expert, d = 1: h_i = 64 v_i exactly (silu(64) is 64, the routing weight 1), with v_i
    set by a scale.  The second product adds h_i with + 1 for v = 1 + 2^-7 - 2^-23, whose bits below the
    second bf16 term are all ones, and with - 1 for v = 1 + 2^-7, which one term holds.  Two rounded
    terms leave at most 2^-17 of each h (two cut-off ones up to 2^-15, all of one sign)."""
    kb = _kb()
    f = 256
    v = torch.full((f,), 1 + 2.0 ** -7, dtype=torch.float64)
    v[::2] -= 2.0 ** -23
    s_in = torch.cat([torch.full((f,), 64.0, dtype=torch.float64), v]).float().reshape(1, 2 * f, 1).cuda()
    ones = torch.ones((1, 2 * f, 1), dtype=torch.int8, device="cuda")
    w_in = kb.bakron_pack(ones, s_in, -8, 7)
    sign = torch.ones((1, 1, f), dtype=torch.int8)
    sign[..., 1::2] = -1
    w_out = kb.bakron_pack(sign.cuda(), torch.ones((1, 1, 1), device="cuda"), -8, 7)
    for dtype in DTYPES:
        x = torch.ones((1, 1), dtype=dtype, device="cuda")
        y = kb.bakron_moe(x, x, w_in, w_out, 1).double().item()
        ref = (64 * v * sign.reshape(-1).double()).sum().item()
        mag = (64 * v).sum().item()
        err = (2.0 ** -17 + 2 * U * (product_depth(f) + 8)) * mag
        # the products' own roundings are bounded apart from h's: the sums here are short and exact to 2^-23
        tight = (2.0 ** -17 + 2.0 ** -22) * mag
        assert abs(y - ref) <= min(err, tight) + HALF_ULP[dtype] * abs(ref) + TINY[dtype]
