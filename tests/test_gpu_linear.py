"""The quantised linear layer on the GPU: bakron_pack, bakron_unpack,
bakron_linear and bakron_linear_grad against the plain 64-bit forms."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, U, bound, product_depth, random_weight, value

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _x(T, n, dtype, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn((T, n), generator=g) * torch.exp(torch.randn(n, generator=g))
    return x.to(dtype).cuda()


def check_linear(y, x, V, dtype):
    xd = x.double()
    ref = xd @ V.T
    b = bound(xd.abs() @ V.abs().T, product_depth(V.shape[1]), dtype, ref)
    assert torch.isfinite(y).all()
    worst = ((y.double() - ref).abs() / b).max().item()
    assert worst <= 1.0, "error %.3g times the bound" % worst


def check_grad(dx, dy, V, dtype):
    yd = dy.double()
    ref = yd @ V
    mag = yd.abs() @ V.abs()
    b = bound(mag, product_depth(V.shape[0], terms=6), dtype, ref)
    if dtype != torch.float32:
        b = b + HALF_ULP[dtype] * mag      # V rounded to dY's type
    worst = ((dx.double() - ref).abs() / b).max().item()
    assert torch.isfinite(dx).all()
    assert worst <= 1.0, "error %.3g times the bound" % worst


@pytest.mark.parametrize("m,n,group,asym,bits", [
    (16, 128, 0, False, 4), (1, 1, 0, True, 4), (17, 130, 32, True, 4), (200, 384, 96, False, 3),
    (130, 1000, 128, True, 2), (8, 33, 32, False, 4), (64, 512, 256, True, 4), (3, 100, 64, False, 2)])
def test_unpack_gives_the_solvers_values(m, n, group, asym, bits):
    """V has the solver's bits: fp32 s times the integer c - z."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, m + n, bits)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    g = group if group and group < n else n
    j = torch.arange(n, device="cuda") // g
    ref = scale[:, j] * (codes.float() - (0 if zero is None else zero[:, j]))
    assert torch.equal(w.unpack(), ref)


def test_unpack_several_matrices():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((3, 20, 70), 32, True, 5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=32)
    j = torch.arange(70, device="cuda") // 32
    assert torch.equal(w.unpack(), scale[..., j] * (codes.float() - zero[..., j]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym", [
    (1, 64, 64, 0, False), (1, 1, 1, 0, True), (1, 1024, 1024, 128, False), (2, 130, 257, 32, True),
    (3, 17, 1111, 96, False), (7, 100, 100, 64, True), (8, 256, 2048, 256, False), (9, 33, 4097, 128, True),
    (15, 500, 640, 32, False), (16, 128, 128, 0, True), (17, 200, 1300, 64, True), (33, 129, 384, 0, False),
    (1, 48, 14336, 128, True), (16, 40, 14336, 32, False), (64, 300, 515, 96, True), (128, 128, 256, 128, False),
    (200, 1000, 1111, 32, True), (257, 512, 1024, 128, False), (1000, 384, 200, 0, True)])
def test_linear(T, m, n, group, asym, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    x = _x(T, n, dtype, m)
    y = kb.bakron_linear(x, w)
    assert y.shape == (T, m) and y.dtype == dtype
    check_linear(y, x, value(codes, scale, zero, group), dtype)
    assert torch.equal(y, kb.bakron_linear(x, w)), "two runs differ"
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 5, 16, 40])
def test_linear_from_unaligned_rows(T, dtype):
    """Activations and outputs at addresses that are multiples of the element
    size only; a guard behind the output stays untouched."""
    kb = _kb()
    m, n = 101, 256
    codes, scale, zero, qmin, qmax = random_weight((m, n), 64, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    base = torch.zeros(T * n + 1, dtype=dtype, device="cuda")
    base[1:] = _x(T, n, dtype, 4).reshape(-1)
    x = base[1:].view(T, n)
    obase = torch.full((T * m + 2,), 7.0, dtype=dtype, device="cuda")
    out = obase[1:-1].view(T, m)
    kb.bakron_linear(x, w, out=out)
    check_linear(out, x, value(codes, scale, zero, 64), dtype)
    assert obase[0] == 7.0 and obase[-1] == 7.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 16, 50])
def test_linear_keeps_nan_and_inf_in_their_rows(T, dtype):
    kb = _kb()
    m, n = 70, 200
    codes, scale, zero, qmin, qmax = random_weight((m, n), 0, False, 8)
    codes[:, 10] = 3
    codes[:, 11] = -2
    w = kb.bakron_pack(codes, scale, qmin, qmax, group=0)
    x = _x(T + 2, n, dtype, 9)
    x[T, 10] = float("nan")
    x[T + 1, 10] = float("inf")
    y = kb.bakron_linear(x, w)
    check_linear(y[:T], x[:T], value(codes, scale, zero, 0), dtype)
    assert torch.isnan(y[T]).all()
    assert (y[T + 1] == float("inf")).all()


def test_linear_no_tokens():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((20, 40), 0, False, 8)
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    assert kb.bakron_linear(torch.empty((0, 40), device="cuda"), w).shape == (0, 20)
    assert kb.bakron_linear_grad(torch.empty((0, 20), device="cuda"), w).shape == (0, 40)


@pytest.mark.parametrize("T", [4, 300])
def test_linear_on_another_stream(T):
    """Work goes to the stream that is asked for, behind what is queued there."""
    kb = _kb()
    m, n = 256, 512
    codes, scale, zero, qmin, qmax = random_weight((m, n), 128, False, 11)
    w = kb.bakron_pack(codes, scale, qmin, qmax, group=128)
    x = _x(T, n, torch.bfloat16, 12)
    want = kb.bakron_linear(x, w)
    s = torch.cuda.Stream()
    late = torch.zeros_like(x)
    out, ws = torch.empty_like(want), kb.linear_workspace(w, T, x.dtype)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        late.copy_(x)
    kb.bakron_linear(late, w, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_linear_in_a_graph():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((128, 256), 32, True, 13)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=32)
    for T in (3, 70):
        x = _x(T, 256, torch.float16, 14)
        out, ws = torch.empty((T, 128), dtype=x.dtype, device="cuda"), kb.linear_workspace(w, T, x.dtype)
        kb.bakron_linear(x, w, out=out, workspace=ws)
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kb.bakron_linear(x, w, out=out, workspace=ws)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_linear_of_a_solved_layer():
    """The solver's codes and V of a layer, used as its weights: the product
    from the packed codes is the product with V."""
    import numpy as np
    kb = _kb()
    from kronecker_factored_gptq_gb300 import workloads as WL
    wl = WL.tiny64(seed=1)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    s = kb.Solver(64, 64, bits=4)
    V, codes = s.solve(put(wl.W), put(wl.A), wl.damp_A, put(wl.B), wl.damp_B)
    w = kb.bakron_pack(codes, s.scale, s.qmin, s.qmax)
    assert torch.equal(w.unpack(), V)
    x = _x(5, 64, torch.float32, 2)
    check_linear(kb.bakron_linear(x, w), x, V.double(), torch.float32)


def test_refusals():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((32, 64), 0, False, 1)
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    x = torch.zeros((4, 64), device="cuda")
    with pytest.raises(ValueError):
        kb.bakron_linear(x.double(), w)
    with pytest.raises(ValueError):
        kb.bakron_linear(x.cpu(), w)
    with pytest.raises(ValueError):
        kb.bakron_linear(x[:, :32], w)
    with pytest.raises(ValueError):
        kb.bakron_linear(torch.zeros((64, 4), device="cuda").T, w)
    with pytest.raises(ValueError):
        kb.bakron_linear(x, w, out=torch.zeros((4, 31), device="cuda"))
    with pytest.raises(ValueError):
        kb.bakron_linear(x, w, out=torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        kb.bakron_linear_grad(x, w)
    with pytest.raises(ValueError):
        kb.bakron_pack(codes, scale, qmin, qmax, group=48)
    bad = codes.clone()
    bad[31, 63] = 9
    with pytest.raises(kb.BakronError) as e:
        kb.bakron_pack(bad, scale, qmin, qmax)
    assert e.value.status == 4
    with pytest.raises(kb.BakronError) as e:
        kb.bakron_pack(codes, scale, qmin, qmax, zero=torch.full_like(scale, 0.5))
    assert e.value.status == 4
    for v in (0.0, -1.0, float("nan"), float("inf")):
        sc = scale.clone()
        sc[5] = v
        with pytest.raises(kb.BakronError) as e:
            kb.bakron_pack(codes, sc, qmin, qmax)
        assert e.value.status == 3
    with pytest.raises(kb.BakronError):
        kb.bakron_pack(codes, scale, -8, 8)      # 17 codes do not fit 4 bits
    two = kb.bakron_pack(torch.stack([codes, codes]), torch.stack([scale, scale]), qmin, qmax)
    with pytest.raises(ValueError):
        kb.bakron_linear(x, two)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym", [
    (1, 64, 64, 0, False), (1, 1, 1, 0, True), (5, 130, 257, 32, True), (16, 17, 1111, 96, False),
    (33, 4097, 100, 64, True), (64, 1000, 300, 128, False), (65, 256, 515, 0, True), (100, 128, 128, 32, False),
    (200, 1111, 1000, 32, True), (257, 1024, 512, 128, False), (333, 520, 1300, 256, True), (1000, 200, 384, 96, False)])
def test_linear_grad(T, m, n, group, asym, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    dy = _x(T, m, dtype, n)
    dx = kb.bakron_linear_grad(dy, w)
    assert dx.shape == (T, n) and dx.dtype == dtype
    check_grad(dx, dy, value(codes, scale, zero, group), dtype)
    assert torch.equal(dx, kb.bakron_linear_grad(dy, w)), "two runs differ"
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_grad_from_unaligned_rows(dtype):
    kb = _kb()
    T, m, n = 40, 256, 101
    codes, scale, zero, qmin, qmax = random_weight((m, n), 64, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    base = torch.zeros(T * m + 1, dtype=dtype, device="cuda")
    base[1:] = _x(T, m, dtype, 4).reshape(-1)
    dy = base[1:].view(T, m)
    obase = torch.full((T * n + 2,), 7.0, dtype=dtype, device="cuda")
    out = obase[1:-1].view(T, n)
    kb.bakron_linear_grad(dy, w, out=out)
    check_grad(out, dy, value(codes, scale, zero, 64), dtype)
    assert obase[0] == 7.0 and obase[-1] == 7.0


def test_linear_grad_against_differences():
    """The loss sum(g * linear(x)) is linear in x, so a central difference of
    the 64-bit form is exact up to its rounding (1e-10 here)."""
    kb = _kb()
    T, m, n = 3, 20, 45
    codes, scale, zero, qmin, qmax = random_weight((m, n), 32, True, 21)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=32)
    V = value(codes, scale, zero, 32)
    x, g = _x(T, n, torch.float32, 1).double(), _x(T, m, torch.float32, 2)
    dx = kb.bakron_linear_grad(g, w)
    mag = g.double().abs() @ V.abs()
    for t in range(T):
        for j in range(n):
            a, b = x.clone(), x.clone()
            a[t, j] += 1e-3
            b[t, j] -= 1e-3
            d = ((g.double() * (a @ V.T)).sum() - (g.double() * (b @ V.T)).sum()) / 2e-3
            tol = bound(mag[t, j], product_depth(m, 6), torch.float32, d) + 1e-9
            assert abs(dx[t, j].item() - d.item()) <= tol


@pytest.mark.parametrize("T,m,n,group,dtype", [
    (64, 8192, 256, 32, torch.bfloat16), (49, 8192, 1000, 96, torch.float16), (50, 19456, 256, 96, torch.bfloat16),
    (33, 8192, 256, 128, torch.bfloat16), (48, 4100, 700, 64, torch.float16), (16, 8192, 1800, 32, torch.float32),
    (16, 19456, 1800, 0, torch.float32), (9, 4096, 4000, 128, torch.float32), (1, 2000, 28000, 64, torch.float32)])
def test_linear_of_many_rows(T, m, n, group, dtype):
    """Enough rows that blocks are as large as they get."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, True, T + m)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    x = _x(T, n, dtype, 1)
    check_linear(kb.bakron_linear(x, w), x, value(codes, scale, zero, group), dtype)
