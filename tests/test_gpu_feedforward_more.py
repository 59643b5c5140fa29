"""The feed-forward calls where a block takes several tiles of an odd number of chunks, two streams
at once, and chains of calls in one graph."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import random_weight, value
from test_gpu_experts import _offsets, check_rows, run
from test_gpu_linear_act import _randn, check_linear_act

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym", [
    (150, 20010, 384, 128, False), (150, 20010, 384, 32, True), (300, 12000, 600, 64, False), (200, 16000, 100, 0, True)])
def test_linear_act_of_many_tiles(T, m, n, group, asym, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + n)
    scale = scale * (10 / n ** 0.5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    x, b, r = _randn((T, n), dtype, m), _randn((m,), torch.float32, 5), _randn((T, m), dtype, 6)
    y, z = kb.bakron_linear_act(x, w, bias=b, act="silu", residual=r, want_pre=True)
    check_linear_act(y, z, x, value(codes, scale, zero, group), b, "silu", r, dtype)
    kb.bakron_async_status()


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,group", [(2500, 384, 128), (2500, 384, 32), (2500, 640, 64), (384, 2500, 0)])
def test_experts_of_many_tiles(m, n, group, dtype, grad):
    kb = _kb()
    counts = [70, 0, 33, 200, 1, 96, 0, 150, 64, 31]
    codes, scale, zero, qmin, qmax = random_weight((len(counts), m, n), group, True, m + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    offsets = _offsets(counts, first=3)
    x = _randn((sum(counts) + 10, m if grad else n), dtype, 4)
    o = offsets.tolist()
    check_rows(run(kb, x, w, offsets, grad, m, n), x, value(codes, scale, zero, group), list(zip(o, o[1:])), dtype, grad)


@pytest.mark.parametrize("dtype", DTYPES)
def test_two_streams_at_once(dtype):
    """Two layers on two streams, each with its workspace, give what they give alone."""
    kb = _kb()
    jobs = []
    for seed, (T, m, n) in enumerate(((500, 700, 512), (90, 3000, 640))):
        codes, scale, zero, qmin, qmax = random_weight((4, m, n), 64, True, seed)
        w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
        x, offsets = _randn((T, n), dtype, seed), _offsets([T // 4] * 4)
        ws = kb.experts_workspace(w, T, dtype)
        want = kb.bakron_experts(x, w, offsets)
        jobs.append((x, w, offsets, ws, torch.zeros_like(want), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for x, w, offsets, ws, out, _, s in jobs:
            kb.bakron_experts(x, w, offsets, out=out, workspace=ws, stream=s)
    torch.cuda.synchronize()
    for *_, out, want, _ in jobs:
        k = want.shape[0] // 4 * 4
        assert torch.equal(out[:k], want[:k])


def test_forward_and_back_in_one_graph():
    """A training pass of the layer captured once, replayed on other tokens and choices."""
    kb = _kb()
    T, d, f, E, k, dtype = 96, 128, 192, 6, 2, torch.bfloat16
    ci, si, _, qmin, qmax = random_weight((E, 2 * f, d), 64, False, 1)
    co, so, _, _, _ = random_weight((E, d, f), 64, False, 2)
    w_in, w_out = kb.bakron_pack(ci, si, qmin, qmax, group=64), kb.bakron_pack(co, so, qmin, qmax, group=64)
    x, dy = _randn((T, d), dtype, 1), _randn((T, d), dtype, 2)
    weight = torch.full((T, k), 0.5, device="cuda")
    choice = torch.randint(0, E, (T, k), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    rows, z, h, o = (torch.zeros((T * k, c), dtype=dtype, device="cuda") for c in (d, 2 * f, f, d))

    def step():
        offsets, place = kb.bakron_sort_tokens(choice, E)
        kb.bakron_dispatch(x, place, out=rows)
        kb.bakron_experts(rows, w_in, offsets, out=z)
        kb.bakron_act(z, "silu", gated=True, out=h)
        kb.bakron_experts(h, w_out, offsets, out=o)
        y = kb.bakron_combine(o, place, weight)
        do, dweight = kb.bakron_combine_grad(dy, o, place, weight)
        dh = kb.bakron_experts_grad(do, w_out, offsets)
        dz, _ = kb.bakron_act_grad(dh, z, "silu", gated=True)
        dx = kb.bakron_combine(kb.bakron_experts_grad(dz, w_in, offsets), place)
        return y, dx, dweight

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for seed in (3, 4):
        x.copy_(_randn((T, d), dtype, seed))
        choice.copy_(torch.randint(0, E, (T, k), device="cuda", generator=torch.Generator("cuda").manual_seed(seed)))
        want = [t.clone() for t in step()]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    kb.bakron_async_status()
