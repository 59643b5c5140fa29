"""bakron_linear_act, bakron_act and bakron_act_grad against the plain 64-bit forms."""

import pytest

torch = pytest.importorskip("torch")

from _feedforward_helpers import ACTS, activation, check, rounded, small
from _layer_helpers import HALF_ULP, U, product_depth, random_weight, value

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed, spread=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (spread * torch.randn(shape, generator=g)).to(dtype).cuda()


def check_linear_act(y, pre, x, V, bias, act, residual, dtype):
    xd = x.double()
    z, mag = xd @ V.T, xd.abs() @ V.abs().T
    ez = 2 * U * product_depth(V.shape[1]) * mag
    if bias is not None:
        z = z + bias.double()
        ez = ez + U * (z.abs() + ez)
    if pre is not None:
        check(pre, z, rounded(ez, z, dtype), "pre")
    a, _, ea, _ = activation(z, act)
    err = 1.13 * ez + ea + 1e-3 * ea            # no slope is above 1.13
    if residual is not None:
        a = a + residual.double()
        err = err + U * (a.abs() + err)
    check(y, a, rounded(err, a, dtype), "y")


# each kernel (few, tens and many tokens), whole and split columns, odd sizes
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym,act,bias,residual,pre", [
    (1, 1024, 1024, 128, False, "silu", True, False, False), (1, 1, 1, 0, True, "gelu", True, True, True),
    (3, 17, 1111, 96, False, "gelu_tanh", False, True, False), (8, 256, 2048, 256, False, "relu", True, True, True),
    (9, 33, 4097, 128, True, "silu", False, False, True), (16, 100, 640, 32, False, "gelu", True, False, False),
    (1, 48, 14336, 128, True, "none", True, True, False), (17, 200, 1300, 64, True, "silu", True, True, True),
    (33, 129, 384, 0, False, "gelu", True, False, True), (48, 300, 515, 96, True, "gelu_tanh", True, True, False),
    (64, 2000, 4096, 128, False, "relu", False, True, True), (65, 128, 256, 128, False, "none", True, False, True),
    (200, 1000, 1111, 32, True, "silu", True, True, True), (257, 512, 1024, 128, False, "gelu", True, True, True),
    (1000, 384, 200, 0, True, "gelu_tanh", True, True, False), (70, 128, 8192, 128, False, "silu", True, True, True)])
def test_linear_act(T, m, n, group, asym, act, bias, residual, pre, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m + n)
    scale = scale * (10 / n ** 0.5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    x = _randn((T, n), dtype, m)
    b = _randn((m,), torch.float32, 5) if bias else None
    r = _randn((T, m), dtype, 6) if residual else None
    y, z = kb.bakron_linear_act(x, w, bias=b, act=act, residual=r, want_pre=pre)
    assert y.shape == (T, m) and y.dtype == dtype and (z is None) == (not pre)
    check_linear_act(y, z, x, value(codes, scale, zero, group), b, act, r, dtype)
    again, z2 = kb.bakron_linear_act(x, w, bias=b, act=act, residual=r, want_pre=pre)
    assert torch.equal(y, again) and (z is None or torch.equal(z, z2)), "two runs differ"
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_without_epilogue_it_is_the_linear_layer(T, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((200, 700), 64, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    x = _randn((T, 700), dtype, 4)
    y, z = kb.bakron_linear_act(x, w, want_pre=True)
    assert torch.equal(y, kb.bakron_linear(x, w)) and torch.equal(z, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [2, 16, 40, 130])
def test_linear_act_at_odd_addresses(T, dtype):
    """Every array at a multiple of its element size; what is beside the outputs stays."""
    kb = _kb()
    m, n = 101, 256
    codes, scale, zero, qmin, qmax = random_weight((m, n), 64, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)

    def odd(t, fill=7.0):
        base = torch.full((t.numel() + 2,), fill, dtype=t.dtype, device="cuda")
        base[1:-1] = t.reshape(-1)
        return base, base[1:-1].view(t.shape)

    x, r, b = (odd(t)[1] for t in (_randn((T, n), dtype, 4), _randn((T, m), dtype, 5), _randn((m,), torch.float32, 6)))
    (ob, out), (pb, pre) = (odd(torch.zeros((T, m), dtype=dtype, device="cuda")) for _ in range(2))
    kb.bakron_linear_act(x, w, bias=b, act="silu", residual=r, want_pre=True, out=out, pre=pre)
    check_linear_act(out, pre, x, value(codes, scale, zero, 64), b, "silu", r, dtype)
    for base in (ob, pb):
        assert base[0] == 7.0 and base[-1] == 7.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_act_keeps_nan_and_inf_in_their_rows(T, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((70, 200), 0, False, 8)
    codes[:, 10] = 3
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    x, r = _randn((T + 3, 200), dtype, 9), _randn((T + 3, 70), dtype, 10)
    x[T, 10], x[T + 1, 10], r[T + 2, 4] = float("nan"), float("inf"), float("inf")
    y, z = kb.bakron_linear_act(x, w, act="relu", residual=r, want_pre=True)
    check_linear_act(y[:T], z[:T], x[:T], value(codes, scale, zero, 0), None, "relu", r[:T], dtype)
    assert torch.isnan(y[T]).all() and torch.isnan(z[T]).all()
    assert (y[T + 1] == float("inf")).all()
    assert y[T + 2, 4] == float("inf") and torch.isfinite(y[T + 2, 5:]).all()


@pytest.mark.parametrize("T", [1, 30, 300])
def test_linear_act_in_a_graph_and_on_another_stream(T):
    kb = _kb()
    m, n, dtype = 256, 512, torch.bfloat16
    codes, scale, zero, qmin, qmax = random_weight((m, n), 128, False, 11)
    w = kb.bakron_pack(codes, scale, qmin, qmax, group=128)
    x, r, b = _randn((T, n), dtype, 1), _randn((T, m), dtype, 2), _randn((m,), torch.float32, 3)
    out, ws = torch.zeros((T, m), dtype=dtype, device="cuda"), kb.linear_workspace(w, T, dtype)
    call = lambda **k: kb.bakron_linear_act(x, w, bias=b, act="gelu", residual=r, out=out, workspace=ws, **k)
    want = call()[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    x2 = _randn((T, n), dtype, 7)
    want2 = kb.bakron_linear_act(x2, w, bias=b, act="gelu", residual=r)[0]
    x.copy_(x2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)


# ---------------------------------------------------------------- activations

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,m", [(1, 1), (1, 1024), (3, 7), (37, 1111), (300, 64), (65, 264), (1000, 8), (2, 14336)])
def test_act_and_its_gradient(T, m, act, gated, dtype):
    kb = _kb()
    z, dy = _randn((T, m * (1 + gated)), dtype, T + m, 3.0), _randn((T, m), dtype, 2)
    y = kb.bakron_act(z, act, gated=gated)
    dz, db = kb.bakron_act_grad(dy, z, act, gated=gated, want_bias_grad=True)
    assert y.shape == (T, m) and dz.shape == z.shape and db.shape == (z.shape[1],) and db.dtype == torch.float32
    g, u = z[:, :m].double(), z[:, m:].double() if gated else torch.ones((T, m), dtype=torch.float64, device="cuda")
    d = dy.double()
    a, slope, ea, es = activation(g, act)
    want, err = a * u, (ea + U * a.abs()) * u.abs()
    check(y, want, rounded(err, want, dtype), "y")
    dg, eg = d * u * slope, (d * u).abs() * (es + 2 * U * slope.abs()) + 2.0 ** -125 * (d * u).abs()
    parts, errs = [dg], [eg]
    if gated:
        parts.append(d * a)
        errs.append(d.abs() * (ea + U * a.abs()))
    ref, err = torch.cat(parts, 1), torch.cat(errs, 1)
    check(dz, ref, rounded(err, ref, dtype), "dz")
    # every value passes at most T additions
    check(db, ref.sum(0), err.sum(0) + U * (T + 2) * ref.abs().sum(0) + small(torch.float32), "dbias")
    dz2, none = kb.bakron_act_grad(dy, z, act, gated=gated)
    assert none is None and torch.equal(dz, dz2)
    again = kb.bakron_act_grad(dy, z, act, gated=gated, want_bias_grad=True)
    assert torch.equal(again[1], db), "two runs differ"


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ACTS)
def test_act_grad_is_the_slope_of_act(act, gated):
    """Central differences in fp32, off the corner of relu.  With h = 2^-6 the difference is off by
    h^2 / 6 times the third derivative (at most 3: gelu's is below 1.6, silu's and the tanh form's
    below 2, times |dy u| < 6) and by the rounding of two values of at most 40 over h."""
    kb = _kb()
    z, dy = _randn((40, 60), torch.float32, 1, 2.0).clamp(-5, 5), _randn((40, 30 if gated else 60), torch.float32, 2).clamp(-3, 3)
    z = torch.where(z.abs() < 0.1, torch.full_like(z, 0.5), z)
    dz, _ = kb.bakron_act_grad(dy, z, act, gated=gated)
    h = 2.0 ** -6
    want = torch.zeros_like(z, dtype=torch.float64)
    for j in range(z.shape[1]):
        step = torch.zeros_like(z)
        step[:, j] = h
        up, down = (kb.bakron_act(z + s * step, act, gated=gated).double() for s in (1, -1))
        want[:, j] = ((up - down) / (2 * h) * dy.double()).sum(1)
    assert (dz.double() - want).abs().max().item() <= h * h / 6 * 3 * 15 + 40 * 2.0 ** -20 / h


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_act_at_the_ends_of_the_range(act, dtype):
    """Finite values give finite results, the limits' where the function has them; NaN stays in its
    place, infinities give what the formula gives."""
    kb = _kb()
    top = torch.finfo(dtype).max
    vals = [0.0, -0.0, top, -top, top / 2, -1e4, 1e4, -100.0, 100.0, -30.0, 30.0, torch.finfo(dtype).tiny]
    z = torch.tensor([vals + [float("nan"), float("inf"), -float("inf"), 1.0]], dtype=dtype, device="cuda")
    dy = torch.ones_like(z)
    y = kb.bakron_act(z, act)[0].double()
    dz = kb.bakron_act_grad(dy, z, act)[0][0].double()
    n = len(vals)
    assert torch.isfinite(y[:n]).all() and torch.isfinite(dz[:n]).all()
    big = torch.tensor(vals, dtype=dtype, device="cuda").double()
    for i, v in enumerate(big.tolist()):
        if act != "none" and abs(v) >= 100:
            # |v| exp(-|v|) is below 2^-125 from 100 on
            assert abs(y[i].item() - max(v, 0.0)) <= 2.0 ** -125 and abs(dz[i].item() - (v > 0)) <= 2.0 ** -125, v
    assert torch.isnan(y[n]) and (act == "none" or torch.isnan(dz[n]))
    assert y[n + 1] == float("inf")
    assert torch.isfinite(y[n + 3]) and torch.isfinite(dz[n + 3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
def test_act_at_odd_addresses_and_sums_of_many_rows(dtype, gated):
    kb = _kb()
    T, m = 3000, 33

    def odd(*shape):
        base = torch.full((T * shape[1] + 2,), 7.0, dtype=dtype, device="cuda")
        return base, base[1:-1].view(shape)

    (_, z), (_, dy), (yb, y), (zb, dz) = odd(T, m * (1 + gated)), odd(T, m), odd(T, m), odd(T, m * (1 + gated))
    z.copy_(_randn(z.shape, dtype, 1))
    dy.copy_(_randn(dy.shape, dtype, 2))
    kb.bakron_act(z, "silu", gated=gated, out=y)
    _, db = kb.bakron_act_grad(dy, z, "silu", gated=gated, want_bias_grad=True, out=dz)
    # the same values at even addresses
    want = kb.bakron_act_grad(dy.clone(), z.clone(), "silu", gated=gated, want_bias_grad=True)
    assert torch.equal(y, kb.bakron_act(z.clone(), "silu", gated=gated)) and torch.equal(dz, want[0])
    ref = dz.double().sum(0)
    check(db, ref, (U * (T + 2) + HALF_ULP[dtype] + 40 * U) * dz.double().abs().sum(0) + small(dtype) * T, "dbias")
    for base in (yb, zb):
        assert base[0] == 7.0 and base[-1] == 7.0


def test_no_rows():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((20, 40), 0, False, 8)
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    y, z = kb.bakron_linear_act(torch.empty((0, 40), device="cuda"), w, act="silu", want_pre=True)
    assert y.shape == (0, 20) and z.shape == (0, 20)
    e = torch.empty((0, 20), device="cuda")
    assert kb.bakron_act(e, "silu", gated=True).shape == (0, 10)
    dz, db = kb.bakron_act_grad(e, e, "silu", want_bias_grad=True)
    assert dz.shape == (0, 20) and (db == 0).all()


def test_a_workspace_serves_fewer_rows():
    kb = _kb()
    ws = kb.act_grad_workspace(4000, 128)
    assert ws is not None
    for T in (1, 100, 3999, 4000):
        z, dy = _randn((T, 128), torch.bfloat16, T), _randn((T, 128), torch.bfloat16, 2)
        a = kb.bakron_act_grad(dy, z, "gelu", want_bias_grad=True, workspace=ws)
        b = kb.bakron_act_grad(dy, z, "gelu", want_bias_grad=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
