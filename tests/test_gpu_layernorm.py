"""bakron_layernorm and bakron_layernorm_grad against the plain 64-bit
forms; the gradients also against differences of the 64-bit forward."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, TINY, U

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
EPS = 1e-5
SIZES = [(1, 1), (1, 2), (3, 64), (5, 127), (37, 1111), (9, 1024), (40, 1032), (3, 2048), (700, 512), (2, 4096),
         (3, 8192), (5, 14336), (2, 16384), (2, 16385), (2, 33000), (2000, 100), (1300, 2056)]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _case(T, d, dtype, seed, offset=0.5):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = (torch.randn((T, d), generator=g) * torch.exp(0.5 * torch.randn(d, generator=g)) +
         offset * torch.randn((T, 1), generator=g)).to(dtype).cuda()
    dy = torch.randn((T, d), generator=g).to(dtype).cuda()
    gamma = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    beta = (0.2 * torch.randn(d, generator=g)).cuda()
    return x, dy, gamma, beta


def forward(x, gamma, beta, eps=EPS):
    x = x.double()
    mu = x.mean(1, keepdim=True)
    r = ((x - mu) ** 2).mean(1, keepdim=True).add(eps).rsqrt()
    h = (x - mu) * r
    y = h if gamma is None else h * gamma.double()
    return (y if beta is None else y + beta.double()), mu, r, h


def backward(dy, x, gamma, eps=EPS):
    _, mu, r, h = forward(x, None, None, eps)
    dy = dy.double()
    a = dy if gamma is None else dy * gamma.double()
    dx = r * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0), h, r, a


# Depth of a sum over the d columns of a row: a thread's elements, the
# shuffles and the warps, never more than 64 + 5 + 32 for rows in registers
# and d / 1024 + 37 for longer ones.
def _depth(d):
    return 101 + d / 1024


def check_forward(y, mean, rstd, x, gamma, beta, dtype):
    ref, mu, r, h = forward(x, gamma, beta)
    d = x.shape[1]
    xd = x.double()
    e_mu = 2 * U * _depth(d) * xd.abs().mean(1, keepdim=True)            # absolute error of mu
    assert ((mean.double()[:, None] - mu).abs() <= e_mu + TINY[torch.float32]).all()
    dev = (xd - mu).abs() + e_mu
    # relative error of r: half of the variance's, which a shift of mu moves only to second order
    e_r = 0.5 * (2 * U * (_depth(d) + 4) + e_mu ** 2 * r ** 2) + 4 * U
    assert ((rstd.double()[:, None] - r).abs() <= e_r * r).all()
    g = torch.ones_like(xd[:1]) if gamma is None else gamma.double().abs()
    b = torch.zeros_like(xd[:1]) if beta is None else beta.double().abs()
    err = (e_mu * r + (h.abs() + e_mu * r) * (e_r + 6 * U)) * g + 2 * U * (h.abs() * g + b)
    tol = err + HALF_ULP[dtype] * (ref.abs() + err) + TINY[dtype]
    worst = ((y.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "error %.3g times the bound" % worst


def check_backward(dx, dgamma, dbeta, dy, x, gamma, mean, rstd, dtype):
    ref, rg, rb, h, r, a = backward(dy, x, gamma)
    T, d = x.shape
    xd = x.double()
    _, mu, _, _ = forward(x, None, None)
    e_mu = 2 * U * _depth(d) * xd.abs().mean(1, keepdim=True)
    e_r = 0.5 * (2 * U * (_depth(d) + 4) + e_mu ** 2 * r ** 2) + 4 * U
    e_h = e_mu * r + (h.abs() + e_mu * r) * (e_r + 4 * U)               # absolute error of h
    m1, m2 = a.abs().mean(1, keepdim=True), (a * h).abs().mean(1, keepdim=True)
    e1 = 2 * U * (_depth(d) + 2) * m1
    e2 = 2 * U * (_depth(d) + 4) * m2 + (a.abs() * e_h).mean(1, keepdim=True)
    err = r * (4 * U * (a.abs() + m1 + h.abs() * m2) + e1 + h.abs() * e2 + e_h * m2) * 1.01 + e_r * ref.abs() + \
        e_r * r * (a.abs() + m1 + h.abs() * m2)
    tol = err + HALF_ULP[dtype] * (ref.abs() + err) + TINY[dtype]
    worst = ((dx.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "dx: error %.3g times the bound" % worst
    if dgamma is not None:
        # a column's sum over rows: at worst one addition per row of a block, then the join
        depth = T / 100 + 200
        dd = dy.double().abs()
        tg = (2 * U * depth * (dd * h.abs()).sum(0) + (dd * e_h).sum(0)) * 1.01 + TINY[torch.float32]
        tb = 2 * U * depth * dd.sum(0) + TINY[torch.float32]
        assert ((dgamma.double() - rg).abs() <= tg).all()
        assert ((dbeta.double() - rb).abs() <= tb).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", SIZES)
def test_forward_and_backward(T, d, dtype):
    kb = _kb()
    x, dy, gamma, beta = _case(T, d, dtype, T + d)
    y, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    check_forward(y, mean, rstd, x, gamma, beta, dtype)
    got = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd)
    check_backward(*got, dy, x, gamma, mean, rstd, dtype)
    again = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "two runs differ"


@pytest.mark.parametrize("d", [96, 1111, 2048, 40000])
def test_without_parameters_or_weight_gradients(d):
    kb = _kb()
    x, dy, _, _ = _case(6, d, torch.float32, d)
    y, mean, rstd = kb.bakron_layernorm(x)
    check_forward(y, mean, rstd, x, None, None, torch.float32)
    dx, dg, db = kb.bakron_layernorm_grad(dy, x, None, mean, rstd, want_weight_grads=False)
    assert dg is None and db is None
    check_backward(dx, None, None, dy, x, None, mean, rstd, torch.float32)
    y2, m2, r2 = kb.bakron_layernorm(x, want_stats=False)
    assert m2 is None and r2 is None and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_unaligned_rows(dtype):
    kb = _kb()
    T, d = 5, 1024
    x, dy, gamma, beta = _case(T, d, dtype, 3)

    def off(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    x, dy, gamma, beta = off(x), off(dy), off(gamma), off(beta)
    y, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    check_forward(y, mean, rstd, x, gamma, beta, dtype)
    check_backward(*kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd), dy, x, gamma, mean, rstd, dtype)


def test_large_mean_keeps_the_variance():
    """Rows whose mean is 1000 standard deviations: the variance comes from
    the deviations, so it keeps its digits."""
    kb = _kb()
    x, dy, gamma, beta = _case(4, 3000, torch.float32, 5, offset=0.0)
    x = x + 1000.0
    y, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    check_forward(y, mean, rstd, x, gamma, beta, torch.float32)


def test_constant_rows_and_bad_values():
    kb = _kb()
    for d in (64, 1111, 4096):
        x = torch.full((3, d), 2.0, device="cuda")
        x[1] = torch.randn(d, device="cuda")
        x[2, d // 2] = float("nan")
        y, mean, rstd = kb.bakron_layernorm(x)
        assert (y[0] == 0).all()
        assert torch.isfinite(y[1]).all() and torch.isnan(y[2]).all()


@pytest.mark.parametrize("T,d", [(2, 5), (3, 40)])
def test_gradient_against_differences(T, d):
    """The loss sum(w * y): its gradients against central differences of the
    64-bit forward (step 1e-4: truncation about 1e-8, rounding about 1e-12)."""
    kb = _kb()
    x, w, gamma, beta = _case(T, d, torch.float32, 17)
    _, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    dx, dg, db = kb.bakron_layernorm_grad(w, x, gamma, mean, rstd)
    loss = lambda x_, g_, b_: (w.double() * forward(x_, g_, b_)[0]).sum()
    step = 1e-4

    def diff(which, i):
        a = [x.double().clone(), gamma.double().clone(), beta.double().clone()]
        b = [t.clone() for t in a]
        a[which].view(-1)[i] += step
        b[which].view(-1)[i] -= step
        return ((loss(*a) - loss(*b)) / (2 * step)).item()

    for which, got in ((0, dx), (1, dg), (2, db)):
        for i in range(got.numel()):
            ref = diff(which, i)
            assert abs(got.reshape(-1)[i].item() - ref) <= 2e-5 * max(1.0, abs(ref)) + 2e-6


def test_no_rows():
    kb = _kb()
    x = torch.empty((0, 24), device="cuda")
    y, mean, rstd = kb.bakron_layernorm(x)
    dx, dg, db = kb.bakron_layernorm_grad(x, x, None, mean, rstd)
    assert y.shape == (0, 24) and dx.shape == (0, 24)
    assert (dg == 0).all() and (db == 0).all()


def test_refusals():
    kb = _kb()
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError):
        kb.bakron_layernorm(x, gamma=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        kb.bakron_layernorm(x, gamma=torch.ones(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        kb.bakron_layernorm(x.T)
    with pytest.raises(kb.BakronError):
        kb.bakron_layernorm(x, eps=-1.0)
    _, mean, rstd = kb.bakron_layernorm(x)
    with pytest.raises(ValueError):
        kb.bakron_layernorm_grad(x.bfloat16(), x, None, mean, rstd)
    with pytest.raises(ValueError):
        kb.bakron_layernorm_grad(x, x, None, mean[:3], rstd)
    with pytest.raises(ValueError):
        kb.bakron_layernorm_grad(x, x, None, mean, rstd, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (9, 130), (700, 37), (40, 255), (30, 1023), (5, 1026),
                                 (400, 1111), (20, 2049), (7, 4100), (9, 9999), (3, 14335)])
@pytest.mark.parametrize("offsets", [(0, 0, 0), (1, 3, 5), (6, 4, 0)])
def test_rows_of_any_alignment(T, d, offsets, dtype):
    """Inputs and outputs at different places inside 16 bytes, NaN around the
    inputs (nothing of them may count), guards around the outputs."""
    kb = _kb()
    x, dy, gamma, beta = _case(T, d, dtype, T + d)

    def put(t, k, pad):
        b = torch.full((t.numel() + 24,), pad, dtype=t.dtype, device="cuda")
        v = b[8 + k:8 + k + t.numel()].view(t.shape)
        v.copy_(t)
        return b, v

    _, x = put(x, offsets[0], float("nan"))
    _, dy = put(dy, offsets[1], float("nan"))
    ybuf, y = put(x, offsets[2], 7.0)
    dbuf, dx = put(x, offsets[1], 7.0)
    _, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS, out=y)
    check_forward(y, mean, rstd, x, gamma, beta, dtype)
    _, dgamma, dbeta = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd, out=dx)
    check_backward(dx, dgamma, dbeta, dy, x, gamma, mean, rstd, dtype)
    for buf, v, k in ((ybuf, y, offsets[2]), (dbuf, dx, offsets[1])):
        assert (buf[:8 + k] == 7).all() and (buf[8 + k + v.numel():] == 7).all()


@pytest.mark.parametrize("d", [28000, 28700, 32768])
def test_fp32_rows_near_the_shared_memory_limit(d):
    kb = _kb()
    x, dy, gamma, beta = _case(3, d, torch.float32, d)
    y, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    check_forward(y, mean, rstd, x, gamma, beta, torch.float32)
    check_backward(*kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd), dy, x, gamma, mean, rstd, torch.float32)


@pytest.mark.parametrize("d", [64, 1000, 1111])
def test_a_workspace_serves_fewer_rows(d):
    kb = _kb()
    ws = kb.layernorm_grad_workspace(400, d)
    for T in (400, 200, 150, 9, 1):
        assert kb.layernorm_grad_workspace_size(T, d) <= ws.numel()
        x, dy, gamma, beta = _case(T, d, torch.float32, T)
        _, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
        got = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd, workspace=ws)
        check_backward(*got, dy, x, gamma, mean, rstd, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", [(152, 300), (153, 300), (150, 1111), (100, 4096), (31, 8000), (152, 5001), (40, 10240),
                                 (300, 10000), (200, 9500)])
def test_few_rows_and_blocks_of_several_sizes(T, d, dtype):
    kb = _kb()
    x, dy, gamma, beta = _case(T, d, dtype, T * d)
    y, mean, rstd = kb.bakron_layernorm(x, gamma, beta, EPS)
    check_forward(y, mean, rstd, x, gamma, beta, dtype)
    got = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd)
    check_backward(*got, dy, x, gamma, mean, rstd, dtype)
    again = kb.bakron_layernorm_grad(dy, x, gamma, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
