"""Calls on another stream that allocate for themselves, with the stream held up while the current
one takes memory and writes it."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import random_weight

pytestmark = pytest.mark.gpu


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(*shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape))).cuda()


def calls(kb):
    """name: call of a fresh input on a stream, all fp32, so that each takes a workspace."""
    T, m, n, E = 90, 200, 130, 3
    codes, scale, zero, qmin, qmax = random_weight((m, n), 64, True, 1)
    w = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    codes, scale, zero, qmin, qmax = random_weight((E, m, n), 64, True, 2)
    we = kb.bakron_pack(codes, scale, qmin, qmax, zero=zero, group=64)
    offsets = torch.tensor([0, 40, 40, T], dtype=torch.int32, device="cuda")
    x, y = _randn(T, n), _randn(T, m)
    return dict(
        linear=(x, lambda t, s: kb.bakron_linear(t, w, stream=s)),
        linear_act=(x, lambda t, s: kb.bakron_linear_act(t, w, act="gelu", want_pre=True, stream=s)),
        linear_grad=(y, lambda t, s: kb.bakron_linear_grad(t, w, stream=s)),
        experts=(x, lambda t, s: kb.bakron_experts(t, we, offsets, stream=s)),
        experts_grad=(y, lambda t, s: kb.bakron_experts_grad(t, we, offsets, stream=s)),
        act_grad=(y, lambda t, s: kb.bakron_act_grad(t, t, "silu", want_bias_grad=True, stream=s)),
        norm_grad=(x, lambda t, s: kb.bakron_layernorm_grad(t, t, None, *kb.bakron_layernorm(t, stream=s)[1:], stream=s)))


@pytest.mark.parametrize("name", ["linear", "linear_act", "linear_grad", "experts", "experts_grad", "act_grad", "norm_grad"])
def test_memory_is_the_calls_own(name):
    kb = _kb()
    given, call = calls(kb)[name]
    flat = lambda r: [t.clone() for t in (r if isinstance(r, tuple) else (r,)) if t is not None]
    want = flat(call(given, None))
    for _ in range(3):
        s = torch.cuda.Stream()
        fresh = given.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)           # some 10 ms
        got = call(fresh, s)
        del fresh
        # every size the call may have let go, written by the current stream before the call runs
        junk = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(5, 18) for _ in range(4)]
        junk += [torch.full_like(given, float("nan")) for _ in range(4)]
        torch.cuda.current_stream().wait_stream(s)
        got = flat(got)
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    kb.bakron_async_status()


def test_in_a_graph_with_a_side_stream():
    """Two calls side by side in one graph, the second on a stream of its own, without outputs of the caller's."""
    kb = _kb()
    jobs = calls(kb)
    (x, linear), (y, grad) = jobs["linear"], jobs["linear_grad"]
    want = linear(x, None).clone(), grad(y, None).clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        a = linear(x, None)
        b = grad(y, s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    kb.bakron_async_status()
