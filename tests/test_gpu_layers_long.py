"""Calls that keep the GPU busy for longer than a bounded wait's budget (about
0.2 s): the budget is a step's, not the call's, so they end without a status."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


@pytest.mark.parametrize("grad,T,m,n", [(False, 131072, 28672, 28672), (True, 98304, 24576, 24576)])
def test_a_long_call_is_no_timeout(grad, T, m, n):
    """fp32, 2.2e14 and 1.2e14 operations.  Whole numbers below 2^24
    throughout, so the result is exact."""
    kb = _kb()
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-8, 8, (m, n), generator=g, dtype=torch.int8, device="cuda")
    w = kb.bakron_pack(codes, torch.ones((m, 1), device="cuda"), -8, 7)
    x = torch.randint(-8, 9, (T, m if grad else n), generator=g, dtype=torch.int8, device="cuda").float()
    kb.bakron_async_status()
    ws = kb.linear_workspace(w, T, x.dtype, grad=grad)
    out = torch.empty((T, n if grad else m), device="cuda")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    (kb.bakron_linear_grad if grad else kb.bakron_linear)(x, w, out=out, workspace=ws)
    b.record()
    b.synchronize()
    assert a.elapsed_time(b) > 300, "too short to show anything: %.0f ms" % a.elapsed_time(b)
    kb.bakron_async_status()
    rows = torch.tensor([0, 1, 127, T // 2 + 5, T - 1], device="cuda")
    V = codes.double()
    assert torch.equal(out[rows].double(), x[rows].double() @ (V if grad else V.T))
