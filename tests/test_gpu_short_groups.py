"""Groups shorter than 128 columns where the tokens' tiles are cut in different ways: units of a chunk that one
set of epilogue warps takes or two in turn, a tile or several per block, odd numbers of chunks, clusters
of up to eight blocks."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import bound, product_depth, random_weight, value
from test_gpu_clusters import graph_time
from test_gpu_linear_act import check_linear_act

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# few columns, so that one set is as good; many, so that two are; 128 and 512 tokens, where tiles of 128 save a
# tile or a round; rows for clusters of one to eight, and for two rounds of blocks
SIZES = [(33, 130, 900), (65, 257, 2600), (96, 300, 2050), (97, 1000, 1537), (128, 5000, 2200), (129, 520, 4100), (40, 1792, 2100),
         (70, 128, 4500), (400, 5120, 1400), (512, 9728, 1400)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group,asym", [(32, True), (64, False), (64, True), (96, False), (192, True)])
@pytest.mark.parametrize("T,m,n", SIZES)
def test_products(T, m, n, group, asym, dtype):
    """The product alone and with its epilogue; the sum's bound is the linear layer's."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m + n)
    scale = scale * (10 / n ** 0.5)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    x = _randn((T, n), dtype, m)
    xd = x.double()
    ref, mag = xd @ V.T, xd.abs() @ V.abs().T
    y = kb.bakron_linear(x, w)
    assert ((y.double() - ref).abs() <= bound(mag, product_depth(n), dtype, ref)).all()
    assert torch.equal(y, kb.bakron_linear(x, w)), "two runs differ"
    b, r = _randn((m,), torch.float32, 5), _randn((T, m), dtype, 6)
    y, z = kb.bakron_linear_act(x, w, bias=b, act="silu", residual=r, want_pre=True)
    check_linear_act(y, z, x, V, b, "silu", r, dtype)
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("group", [32, 64, 96])
@pytest.mark.parametrize("counts,m,n", [([128, 0, 127, 1, 40], 300, 2200), ([300, 129, 64], 4000, 1400), ([9, 3], 128, 4500),
                                        ([128] * 4, 4864, 1400), ([600, 1, 500], 5120, 700)])
def test_experts(counts, m, n, group, dtype):
    kb = _kb()
    E, R = len(counts), sum(counts) + 3
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), group, True, R)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    V = value(codes, scale, zero, group)
    offsets = torch.tensor([2 + sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    x = _randn((R, n), dtype, m)
    out = torch.full((R, m), 7.0, dtype=dtype, device="cuda")
    kb.bakron_experts(x, w, offsets, out=out)
    kb.bakron_async_status()
    o = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(o, o[1:])):
        xd = x[lo:hi].double()
        ref, mag = xd @ V[e].T, xd.abs() @ V[e].abs().T
        assert ((out[lo:hi].double() - ref).abs() <= bound(mag, product_depth(n), dtype, ref)).all(), "expert %d" % e
    assert (out[:2] == 7.0).all() and (out[o[-1]:] == 7.0).all()


@pytest.mark.parametrize("m,n,most", [(8192, 8192, 1.3), (4096, 4096, 1.25)])
def test_a_third_more_tokens_take_no_second_tile(m, n, most):
    """128 tokens against 96 in groups of 64: tiles of 128 take 1.09 and 1.05 times as long, two tiles
    of 64 took 1.58 and 1.31."""
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), 64, True, 1)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    t = {}
    for T in (96, 128):
        x, out = _randn((T, n), torch.bfloat16, T), torch.empty((T, m), dtype=torch.bfloat16, device="cuda")
        ws = kb.linear_workspace(w, T, torch.bfloat16)
        t[T] = graph_time(lambda: kb.bakron_linear(x, w, out=out, workspace=ws))
    assert t[128] < most * t[96], t
