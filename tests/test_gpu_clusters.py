"""The product for many tokens where few tiles share their columns among up to eight blocks of a cluster."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import bound, product_depth, random_weight, value
from test_gpu_linear_act import check_linear_act

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group", [(65, 1, 2100, 0), (96, 128, 16384, 128), (100, 300, 4097, 128), (192, 640, 2048, 0),
                                         (66, 1792, 2048, 128), (70, 2000, 2300, 256), (130, 257, 8190, 0)])
def test_linear(T, m, n, group, dtype):
    """One to more tiles than clusters of eight fit at once, even and odd shares of the columns."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, True, T + m)
    scale = scale * (10 / n ** 0.5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    x = _randn((T, n), dtype, m)
    xd = x.double()
    ref, mag = xd @ V.T, xd.abs() @ V.abs().T
    y = kb.bakron_linear(x, w)
    assert ((y.double() - ref).abs() <= bound(mag, product_depth(n), dtype, ref)).all()
    assert torch.equal(y, kb.bakron_linear(x, w)), "two runs differ"
    r = _randn((T, m), dtype, 6)
    y, z = kb.bakron_linear_act(x, w, act="gelu", residual=r, want_pre=True)
    check_linear_act(y, z, x, V, None, "gelu", r, dtype)
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts", [[1, 0], [5, 3], [0, 40, 0], [2, 2, 2]])
def test_experts(counts, dtype):
    """Experts whose rows are known on the device alone: clusters without a tile among them."""
    kb = _kb()
    E, R, m, n = len(counts), sum(counts) + 2, 200, 4100
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), 128, True, R)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=128)
    V = value(codes, scale, zero, 128)
    offsets = torch.tensor([1 + sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    x, out = _randn((R, n), dtype, 3), torch.full((R, m), 7.0, dtype=dtype, device="cuda")
    kb.bakron_experts(x, w, offsets, out=out)
    kb.bakron_async_status()
    o = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(o, o[1:])):
        xd = x[lo:hi].double()
        ref, mag = xd @ V[e].T, xd.abs() @ V[e].abs().T
        assert ((out[lo:hi].double() - ref).abs() <= bound(mag, product_depth(n), dtype, ref)).all(), "expert %d" % e
    assert (out[0] == 7.0).all() and (out[o[-1]:] == 7.0).all()


def graph_time(call, calls=20):
    """Microseconds of a call in a graph of some, the best of twelve replays."""
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(calls):
            call()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    best = float("inf")
    for _ in range(12):
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


def test_eight_blocks_share_a_long_tile():
    """96 tokens of one tile, 16384 columns against 2048: 1.93 times as long in clusters of eight, 2.64 in
    clusters of four."""
    kb = _kb()
    t = {}
    for n in (2048, 16384):
        codes, scale, zero, qmin, qmax = random_weight((128, n), 128, False, 1)
        w = kb.bakron_pack(codes, scale, qmin, qmax, group=128)
        x, out = _randn((96, n), torch.bfloat16, n), torch.empty((96, 128), dtype=torch.bfloat16, device="cuda")
        ws = kb.linear_workspace(w, 96, torch.bfloat16)
        t[n] = graph_time(lambda: kb.bakron_linear(x, w, out=out, workspace=ws))
    assert t[16384] < 2.25 * t[2048], t
