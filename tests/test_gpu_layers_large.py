"""The quantised layers where a block takes several tiles or items: sizes at
which the kernels' loops, rings and barriers go round more than once."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, TINY, random_weight, value
from test_gpu_linear import _x, check_grad, check_linear
from test_gpu_moe import _layer, _tokens, check, reference

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


# tokens per tile of the 16-bit forward: 192, 160, 128 (with groups under 128 at most that); several tiles a
# block, but for the last two shapes
LINEAR = [(2048, 8192, 512, 128, False), (2048, 4096, 1000, 0, True), (1000, 8200, 300, 64, True),
          (1500, 4097, 515, 96, False), (700, 14336, 260, 256, True), (2048, 2100, 256, 32, True),
          (128, 19456, 384, 128, False), (65, 14336, 4096, 64, True)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,m,n,group,asym", LINEAR)
def test_linear_with_several_tiles_a_block(T, m, n, group, asym, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + m)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    x = _x(T, n, dtype, n)
    y = kb.bakron_linear(x, w)
    check_linear(y, x, value(codes, scale, zero, group), dtype)
    assert torch.equal(y, kb.bakron_linear(x, w))
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n,m,group,asym", LINEAR)
def test_linear_grad_with_several_tiles_a_block(T, m, n, group, asym, dtype):
    kb = _kb()
    codes, scale, zero, qmin, qmax = random_weight((m, n), group, asym, T + n)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=group)
    dy = _x(T, m, dtype, n)
    dx = kb.bakron_linear_grad(dy, w)
    check_grad(dx, dy, value(codes, scale, zero, group), dtype)
    assert torch.equal(dx, kb.bakron_linear_grad(dy, w))
    kb.bakron_async_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k,d,f,group,asym", [
    (1, 8, 2, 1500, 3000, 128, True), (4, 8, 2, 1500, 3000, 32, False), (16, 8, 2, 1024, 4096, 128, False),
    (16, 8, 2, 1500, 3001, 0, True), (32, 8, 2, 1500, 3000, 64, True), (32, 5, 3, 4100, 2000, 256, False),
    (12, 60, 4, 640, 1200, 96, True), (3, 4, 4, 8192, 2600, 128, True)])
def test_moe_with_several_items_a_block(T, E, k, d, f, group, asym, dtype):
    kb = _kb()
    w_in, w_out, Vi, Vo = _layer(E, d, f, group, asym, T + E + d)
    x, r = _tokens(T, E, d, dtype, f)
    y = kb.bakron_moe(x, r, w_in, w_out, k)
    check(y, x, r, Vi, Vo, k, True, dtype)
    assert torch.equal(y, kb.bakron_moe(x, r, w_in, w_out, k))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,d,f,group", [(32, 2, 1500, 3000, 128), (32, 1, 1500, 2000, 32), (31, 3, 2100, 1600, 0),
                                           (16, 2, 4096, 1000, 64)])
def test_moe_with_all_tokens_at_one_expert(T, k, d, f, group, dtype):
    """Expert 2 is every token's first choice: its tokens are the most that a
    block can meet, staged in parts.  Activations of one sign make large
    results: past the largest fp16 they are infinite."""
    kb = _kb()
    w_in, w_out, Vi, Vo = _layer(6, d, f, group, True, T + d)
    x, r = _tokens(T, 6, d, dtype, f)
    x = x.abs() + 0.1
    r[2] = 2.0 / d ** 0.5
    y = kb.bakron_moe(x, r, w_in, w_out, k)
    ref, err, ids = reference(x, r, Vi, Vo, k, True)
    assert all(i[0] == 2 for i in ids)
    tol = 1.01 * err + HALF_ULP[dtype] * (ref.abs() + err) + TINY[dtype]
    big = torch.finfo(dtype).max
    out = ref.abs() - tol > big
    assert (y[out].double() == ref[out].sign() * float("inf")).all()
    ok = ~out & (ref.abs() + tol < big)
    assert ok.float().mean() > 0.9 and ((y.double() - ref).abs()[ok] <= tol[ok]).all()
    assert torch.equal(y, kb.bakron_moe(x, r, w_in, w_out, k))
