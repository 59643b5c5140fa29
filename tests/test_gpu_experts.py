"""The experts' products over sorted rows, both ways, against the plain 64-bit forms, and the
steps of a mixture-of-experts layer together, forward and back."""

import pytest

torch = pytest.importorskip("torch")

from _feedforward_helpers import places, random_choices
from _layer_helpers import HALF_ULP, U, bound, product_depth, random_weight, value

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _offsets(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")


def check_rows(y, x, V, bounds, dtype, grad):
    """bounds: (begin, end) of every expert; the other rows are still 7."""
    other = torch.ones(len(x), dtype=torch.bool, device="cuda")
    for e, (lo, hi) in enumerate(bounds):
        if lo == hi:
            continue
        other[lo:hi] = False
        xd, v = x[lo:hi].double(), V[e] if grad else V[e].T
        ref, mag = xd @ v, xd.abs() @ v.abs()
        b = bound(mag, product_depth(v.shape[0], terms=6 if grad else 3), dtype, ref)
        if grad and dtype != torch.float32:
            b = b + HALF_ULP[dtype] * mag      # V rounded to dY's type
        got = y[lo:hi]
        assert torch.isfinite(got).all()
        worst = ((got.double() - ref).abs() / b).max().item()
        assert worst <= 1.0, "expert %d: error %.3g times the bound" % (e, worst)
    assert (y[other] == 7.0).all(), "rows of no expert were written"


def run(kb, x, w, offsets, grad, m, n):
    out = torch.full((len(x), n if grad else m), 7.0, dtype=x.dtype, device="cuda")
    fn = kb.bakron_experts_grad if grad else kb.bakron_experts
    fn(x, w, offsets, out=out)
    again = torch.full_like(out, 7.0)
    fn(x, w, offsets, out=again)
    assert torch.equal(out, again), "two runs differ"
    kb.bakron_async_status()
    return out


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,tail,m,n,group,asym", [
    ([1], 0, 1, 1, 0, True), ([0, 1, 0], 2, 17, 130, 32, True), ([3, 0, 40, 1, 0, 200], 5, 130, 257, 64, True),
    ([33, 32, 31, 64, 65, 1], 0, 128, 256, 128, False), ([0, 0, 0], 9, 40, 64, 0, False),
    ([500], 0, 300, 515, 96, True), ([7, 300, 0, 190, 193], 0, 384, 640, 128, False), ([2] * 60, 0, 64, 96, 32, False),
    ([5, 9], 0, 48, 14336, 128, True), ([5, 9], 3, 5000, 96, 0, False), ([100, 1500], 0, 1000, 200, 64, False)])
def test_experts(counts, tail, m, n, group, asym, dtype, grad):
    kb = _kb()
    E = len(counts)
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), group, asym, sum(counts) + m + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    offsets = _offsets(counts)
    x = _randn((sum(counts) + tail, m if grad else n), dtype, m)
    o = offsets.tolist()
    y = run(kb, x, w, offsets, grad, m, n)
    check_rows(y, x, value(codes, scale, zero, group), list(zip(o, o[1:])), dtype, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_thousand_experts(dtype, grad):
    """The largest number of experts, whose table takes the most shared memory."""
    kb = _kb()
    E, m, n = 1024, 40, 130
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), 32, True, 5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=32)
    counts = [(7 * e) % 5 for e in range(E)]
    x = _randn((sum(counts) + 1, m if grad else n), dtype, 6)
    offsets = _offsets(counts)
    o = offsets.tolist()
    check_rows(run(kb, x, w, offsets, grad, m, n), x, value(codes, scale, zero, 32), list(zip(o, o[1:])), dtype, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_that_are_not_ascending_or_outside(dtype, grad):
    """An offset below an earlier one, below 0 or above the rows counts as the nearest that is not."""
    kb = _kb()
    m, n, R = 70, 140, 90
    codes, scale, zero, qmin, qmax = random_weight((6, m, n), 64, True, 9)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    x = _randn((R, m if grad else n), dtype, 1)
    for given, taken in (([-5, 10, 4, 50, 1 << 30, 60, 70], [0, 10, 10, 50, 90, 90, 90]),
                         ([3, 3, 20, -(1 << 31), 21, 88, 89], [3, 3, 20, 20, 21, 88, 89]),
                         ([95, 0, 0, 0, 0, 0, 0], [90] * 7)):
        offsets = torch.tensor(given, dtype=torch.int32, device="cuda")
        check_rows(run(kb, x, w, offsets, grad, m, n), x, value(codes, scale, zero, 64), list(zip(taken, taken[1:])), dtype, grad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_at_odd_addresses(dtype, grad):
    kb = _kb()
    m, n = 101, 256
    codes, scale, zero, qmin, qmax = random_weight((3, m, n), 64, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    offsets = _offsets([10, 0, 45])
    K, N = (m, n) if grad else (n, m)
    base = torch.zeros(60 * K + 1, dtype=dtype, device="cuda")
    base[1:] = _randn((60 * K,), dtype, 4)
    x = base[1:].view(60, K)
    obase = torch.full((60 * N + 2,), 7.0, dtype=dtype, device="cuda")
    out = obase[1:-1].view(60, N)
    (kb.bakron_experts_grad if grad else kb.bakron_experts)(x, w, offsets, out=out)
    check_rows(out, x, value(codes, scale, zero, 64), [(0, 10), (10, 10), (10, 55)], dtype, grad)
    assert obase[0] == 7.0 and obase[-1] == 7.0


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_sums_of_the_gradient(dtype):
    """Chains that are joined through the workspace (fp16: more than 4096 rows of V)."""
    kb = _kb()
    m, n = 9000, 100
    codes, scale, zero, qmin, qmax = random_weight((3, m, n), 0, True, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero)
    counts = [20, 0, 70]
    offsets = _offsets(counts)
    dy = _randn((90, m), dtype, 1)
    check_rows(run(kb, dy, w, offsets, True, m, n), dy, value(codes, scale, zero, 0), [(0, 20), (20, 20), (20, 90)], dtype, True)


@pytest.mark.parametrize("grad", [False, True])
def test_one_expert_is_the_linear_layer(grad):
    """With all rows in one expert the arithmetic is the linear layer's: within its bound of it, and
    at sizes where both take whole columns the same bits."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((1, 2560, 2560), 128, False, 3)
    w = kb.bakron_pack(codes, scale, qmin, qmax, group=128)
    x = _randn((2000, 2560), torch.bfloat16, 4)
    offsets = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    a = (kb.bakron_experts_grad if grad else kb.bakron_experts)(x, w, offsets)
    b = (kb.bakron_linear_grad if grad else kb.bakron_linear)(x, w)
    assert torch.equal(a, b)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_inf_stay_in_their_rows(dtype, grad):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((2, 70, 200), 0, False, 8)
    codes[codes == 0] = 1
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    x = _randn((12, 70 if grad else 200), dtype, 9)
    V = value(codes, scale, zero, 0)
    x[3, 10], x[8, 10] = float("nan"), float("inf")
    out = torch.full((12, 200 if grad else 70), 7.0, dtype=dtype, device="cuda")
    (kb.bakron_experts_grad if grad else kb.bakron_experts)(x, w, _offsets([5, 6]), out=out)
    assert torch.isnan(out[3]).all()
    col = V[1][10] if grad else V[1][:, 10]
    assert torch.equal(out[8].double(), torch.where(col > 0, float("inf"), -float("inf")).double())
    keep = [i for i in range(12) if i not in (3, 8)]
    assert torch.isfinite(out[keep]).all() and (out[11] == 7).all()


def test_no_rows():
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((2, 20, 40), 0, False, 8)
    w = kb.bakron_pack(codes, scale, qmin, qmax)
    o = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert kb.bakron_experts(torch.empty((0, 40), device="cuda"), w, o).shape == (0, 20)
    assert kb.bakron_experts_grad(torch.empty((0, 20), device="cuda"), w, o).shape == (0, 40)


@pytest.mark.parametrize("grad", [False, True])
def test_a_workspace_serves_fewer_rows_and_other_graphs(grad):
    """Two captured graphs on one workspace, replayed in turn, and offsets that change."""
    kb = _kb()
    m, n, dtype = 130, 257, torch.bfloat16
    codes, scale, zero, qmin, qmax = random_weight((4, m, n), 32, True, 8)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=32)
    V = value(codes, scale, zero, 32)
    ws = kb.experts_workspace(w, 300, dtype, grad=grad)
    fn = kb.bakron_experts_grad if grad else kb.bakron_experts
    K, N = (m, n) if grad else (n, m)
    offsets = _offsets([10, 0, 100, 60])
    jobs = []
    for R, seed in ((300, 1), (170, 2)):
        x, out = _randn((R, K), dtype, seed), torch.full((R, N), 7.0, dtype=dtype, device="cuda")
        fn(x, w, offsets, out=out, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn(x, w, offsets, out=out, workspace=ws)
        jobs.append((x, out, g))
    for counts in ([10, 0, 100, 60], [0, 170, 0, 0], [1, 2, 3, 4]):
        offsets.copy_(_offsets(counts))
        o = offsets.tolist()
        for x, out, g in jobs:
            out.fill_(7.0)
            g.replay()
        for x, out, g in jobs:
            check_rows(out, x, V, list(zip(o, o[1:])), dtype, grad)


def test_the_steps_together():
    """A mixture-of-experts layer and all its gradients in steps, against fp64 autograd.  Four products
    lie on the longest way, each off by at most 2 u product_depth < 2^-16 of its magnitude sum, which at
    these sizes is below 2^3 times the largest result: 2^-11 of the largest in all."""
    kb = _kb()
    T, d, f, E, k = 150, 192, 160, 8, 3
    ci, si, zi, qmin, qmax = random_weight((E, 2 * f, d), 64, True, 1)
    co, so, zo, _, _ = random_weight((E, d, f), 32, True, 2)
    si, so = si * 3 / d ** 0.5 * 10, so * 3 / f ** 0.5 * 10
    w_in, w_out = kb.bakron_pack(ci, si, qmin, qmax, zero=zi, group=64), kb.bakron_pack(co, so, qmin, qmax, zero=zo, group=32)
    Vi, Vo = value(ci, si, zi, 64), value(co, so, zo, 32)
    x, dy = _randn((T, d), torch.float32, 3), _randn((T, d), torch.float32, 4)
    choice = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)])
    choice[10:20] = -1                                     # padding
    weight = torch.softmax(_randn((T, k), torch.float32, 5), 1)

    offsets, place = kb.bakron_sort_tokens(choice.cuda(), E)
    rows = kb.bakron_dispatch(x, place)
    z = kb.bakron_experts(rows, w_in, offsets)
    h = kb.bakron_act(z, "silu", gated=True)
    o = kb.bakron_experts(h, w_out, offsets)
    y = kb.bakron_combine(o, place, weight)
    do, dweight = kb.bakron_combine_grad(dy, o, place, weight)
    dh = kb.bakron_experts_grad(do, w_out, offsets)
    dz, _ = kb.bakron_act_grad(dh, z, "silu", gated=True)
    drows = kb.bakron_experts_grad(dz, w_in, offsets)
    dx = kb.bakron_combine(drows, place)
    kb.bakron_async_status()

    xd, wd = x.double().requires_grad_(), weight.double().requires_grad_()
    want = torch.zeros_like(xd)
    for e in range(E):
        t, j = torch.nonzero(choice.cuda() == e, as_tuple=True)
        gu = xd[t] @ Vi[e].T
        want = want.index_add(0, t, wd[t, j, None] * ((torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ Vo[e].T))
    want.backward(dy.double())
    for got, ref in ((y, want.detach()), (dx, xd.grad), (dweight, wd.grad)):
        assert (got.double() - ref).abs().max().item() <= 2.0 ** -11 * ref.abs().max().item()
    assert (y[10:20] == 0).all() and (dx[10:20] == 0).all() and (dweight[10:20] == 0).all()


def test_the_steps_agree_with_the_layer_for_few_tokens():
    """bakron_moe and the steps on the same tokens, with the weights of its routing.  Two products
    and the weights in fp32 on both sides: 2^-11 of the largest, as above."""
    kb = _kb()
    T, d, f, E, k = 20, 256, 96, 8, 2
    ci, si, zi, qmin, qmax = random_weight((E, 2 * f, d), 64, False, 1)
    co, so, zo, _, _ = random_weight((E, d, f), 32, False, 2)
    w_in, w_out = kb.bakron_pack(ci, si, qmin, qmax, group=64), kb.bakron_pack(co, so, qmin, qmax, group=32)
    x, router = _randn((T, d), torch.float32, 3), _randn((E, d), torch.float32, 4) / d ** 0.5
    want = kb.bakron_moe(x, router, w_in, w_out, k)
    top, choice = torch.topk(x.double() @ router.double().T, k, dim=1)
    weight = torch.softmax(top, 1).float()
    offsets, place = kb.bakron_sort_tokens(choice, E)
    h = kb.bakron_act(kb.bakron_experts(kb.bakron_dispatch(x, place), w_in, offsets), "silu", gated=True)
    y = kb.bakron_combine(kb.bakron_experts(h, w_out, offsets), place, weight)
    assert (y - want).abs().max().item() <= 2.0 ** -11 * want.abs().max().item()
