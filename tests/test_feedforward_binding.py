"""What the feed-forward calls of the Python binding refuse, and that they launch on the current
device only.  No GPU: tensors that say where they are (test_layers_device)."""

import pytest

torch = pytest.importorskip("torch")

from test_layers_device import Called, Stream, device, kb, on, weight  # noqa: F401

I32, F32 = torch.int32, torch.float32


def calls(i, workspace=None, stream=Stream(0)):
    """Each call with everything on one device."""
    x, y, rows = on(i, 3, 64), on(i, 3, 32), on(i, 6, 64)
    w, we = weight(i), weight(i, 2)
    place, wt = on(i, 3, 2, dtype=I32), on(i, 3, 2)
    keep = dict(workspace=workspace, stream=stream)
    return dict(
        linear_act=lambda **k: kb.bakron_linear_act(**{**dict(x=x, w=w, act="silu", out=y, **keep), **k}),
        act=lambda **k: kb.bakron_act(**{**dict(z=x, act="silu", gated=True, out=y, stream=stream), **k}),
        act_grad=lambda **k: kb.bakron_act_grad(**{**dict(dy=y, z=x, act="silu", gated=True, out=on(i, 3, 64), **keep), **k}),
        sort=lambda **k: kb.bakron_sort_tokens(**{**dict(choice=place, experts=4, out=(on(i, 5, dtype=I32), on(i, 3, 2, dtype=I32)),
                                                         stream=stream), **k}),
        dispatch=lambda **k: kb.bakron_dispatch(**{**dict(x=x, place=place, weight=wt, out=rows, stream=stream), **k}),
        combine=lambda **k: kb.bakron_combine(**{**dict(rows=rows, place=place, weight=wt, out=x, stream=stream), **k}),
        combine_grad=lambda **k: kb.bakron_combine_grad(**{**dict(dy=x, rows=rows, place=place, weight=wt,
                                                                  out=(on(i, 6, 64), on(i, 3, 2)), stream=stream), **k}),
        experts=lambda **k: kb.bakron_experts(**{**dict(x=rows, w=we, offsets=on(i, 3, dtype=I32), out=on(i, 6, 32), **keep), **k}),
        experts_grad=lambda **k: kb.bakron_experts_grad(**{**dict(dy=on(i, 6, 32), w=we, offsets=on(i, 3, dtype=I32),
                                                                  out=on(i, 6, 64), **keep), **k}))


NAMES = list(calls(0))


@pytest.fixture(autouse=True)
def sizes(monkeypatch):
    monkeypatch.setattr(kb, "_ACT_WS", {})


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device(device, name):  # noqa: F811
    ws = on(0, 4096, dtype=torch.uint8)
    with pytest.raises(Called):
        calls(0, ws)[name]()
    with pytest.raises(ValueError, match="current device"):
        calls(1, on(1, 4096, dtype=torch.uint8))[name]()
    with pytest.raises(ValueError, match="stream"):
        calls(0, ws, Stream(1))[name]()
    device[0] = 1
    with pytest.raises(ValueError, match="current device"):
        calls(0, ws)[name]()


REFUSED = [
    ("linear_act", dict(x=on(0, 3, 63))), ("linear_act", dict(x=on(0, 3, 64, dtype=torch.float64))), ("linear_act", dict(act="swish")),
    ("linear_act", dict(act=None)), ("linear_act", dict(bias=on(0, 31))), ("linear_act", dict(bias=on(0, 32, dtype=torch.bfloat16))),
    ("linear_act", dict(bias=on(1, 32))), ("linear_act", dict(residual=on(0, 2, 32))), ("linear_act", dict(residual=on(1, 3, 32))),
    ("linear_act", dict(residual=on(0, 3, 32, dtype=torch.float16))), ("linear_act", dict(residual=on(0, 3, 64)[:, ::2])),
    ("linear_act", dict(pre=on(0, 3, 32))), ("linear_act", dict(pre=on(0, 3, 31), want_pre=True)), ("linear_act", dict(w=weight(0, 2))),
    ("linear_act", dict(out=on(0, 3, 64))), ("linear_act", dict(w=weight(1))),
    ("act", dict(act="tanh")), ("act", dict(z=on(0, 3, 63))), ("act", dict(z=on(0, 3, 0))), ("act", dict(z=on(0, 64))),
    ("act", dict(z=on(0, 64, 3).T)), ("act", dict(out=on(0, 3, 64))),
    ("act_grad", dict(dy=on(0, 3, 64))), ("act_grad", dict(dy=on(0, 3, 32, dtype=torch.float16))), ("act_grad", dict(act="x")),
    ("act_grad", dict(out=on(0, 3, 32))), ("act_grad", dict(want_bias_grad=True, workspace=on(0, 63, dtype=torch.uint8))),
    ("sort", dict(choice=on(0, 3, 2))), ("sort", dict(choice=on(0, 6, dtype=I32))), ("sort", dict(choice=on(0, 3, 33, dtype=I32))),
    ("sort", dict(choice=on(0, 3, 0, dtype=I32))), ("sort", dict(choice=on(0, 2, 3, dtype=I32).T)), ("sort", dict(experts=0)),
    ("sort", dict(experts=1025)), ("sort", dict(out=(on(0, 4, dtype=I32), on(0, 3, 2, dtype=I32)))),
    ("sort", dict(out=(on(0, 5, dtype=I32), on(0, 3, 2, dtype=torch.int64)))), ("sort", dict(out=(on(1, 5, dtype=I32), on(0, 3, 2, dtype=I32)))),
    ("dispatch", dict(place=on(0, 2, 2, dtype=I32))), ("dispatch", dict(place=on(0, 3, 2, dtype=torch.int64))),
    ("dispatch", dict(place=on(1, 3, 2, dtype=I32))), ("dispatch", dict(place=on(0, 6, dtype=I32))), ("dispatch", dict(place=None)),
    ("dispatch", dict(weight=on(0, 3, 1))), ("dispatch", dict(weight=on(0, 3, 2, dtype=torch.float16))), ("dispatch", dict(weight=on(1, 3, 2))),
    ("dispatch", dict(out=on(0, 6, 63))), ("dispatch", dict(out=on(0, 6))), ("dispatch", dict(out=7)),
    ("dispatch", dict(place=on(0, 3, 4, dtype=I32)[:, ::2])),
    ("combine", dict(place=on(0, 2, 2, dtype=I32))), ("combine", dict(place=3)), ("combine", dict(rows=on(0, 6, 64, dtype=torch.float16))),
    ("combine", dict(weight=on(0, 2, 2))), ("combine", dict(out=on(0, 2, 64))),
    ("combine_grad", dict(weight=None)), ("combine_grad", dict(rows=on(0, 6, 63))), ("combine_grad", dict(rows=on(1, 6, 64))),
    ("combine_grad", dict(out=(on(0, 6, 64), on(0, 3, 1)))), ("combine_grad", dict(out=(on(0, 5, 64), on(0, 3, 2)))),
    ("combine_grad", dict(out=(on(0, 6, 64), None))), ("combine_grad", dict(dy=on(0, 4, 64))),
    ("experts", dict(offsets=on(0, 2, dtype=I32))), ("experts", dict(offsets=on(0, 3, dtype=torch.int64))),
    ("experts", dict(offsets=on(1, 3, dtype=I32))), ("experts", dict(x=on(0, 6, 32))), ("experts", dict(out=on(0, 5, 32))),
    ("experts", dict(w=weight(1, 2))), ("experts", dict(workspace=on(0, 63, dtype=torch.uint8))), ("experts", dict(offsets=None)),
    ("experts_grad", dict(dy=on(0, 6, 64))), ("experts_grad", dict(out=on(0, 6, 32))), ("experts_grad", dict(offsets=on(0, 4, dtype=I32)))]


@pytest.mark.parametrize("i", range(len(REFUSED)))
def test_refusals(device, i):  # noqa: F811
    name, bad = REFUSED[i]
    with pytest.raises(ValueError):
        calls(0, on(0, 4096, dtype=torch.uint8))[name](**bad)


def test_workspace_sizes_are_asked_on_their_device(device):  # noqa: F811
    w = weight(1, 2)
    with pytest.raises(ValueError, match="current device"):
        kb.experts_workspace_size(w, 5, F32)
    device[0] = 1
    assert kb.experts_workspace_size(w, 5, F32) == 64
    assert kb.experts_workspace_size(w, 5, F32, grad=True) == 64
    assert kb.act_grad_workspace_size(5, 64) == 64 and (5, 64, 1) in kb._ACT_WS
