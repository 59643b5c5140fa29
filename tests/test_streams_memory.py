"""A call on another stream than the current one: what it allocates is that stream's memory, and
what it was given stays until the call has run.  Memory of the current stream's pool would be
handed out again in that stream's order, while the call still reads and writes it.  No GPU: tensors,
streams and a library that say what happens to them."""

import types

import pytest

torch = pytest.importorskip("torch")

from test_layers_device import Library, Placed, kb

I32, F32, I8, U8 = torch.int32, torch.float32, torch.int8, torch.uint8


class Stream:
    device_index = 0

    def __init__(self, handle):
        self.cuda_stream = handle


CURRENT, SIDE = Stream(7), Stream(8)


class Noted(Placed):
    """A tensor that keeps whose memory it has and which streams use it."""

    pool, users = None, ()

    def record_stream(self, stream):
        self.users = self.users + (stream.cuda_stream,)


class Quiet(Library):
    """The library: sizes as in Library, every call succeeds."""

    def __getattr__(self, name):
        if name.endswith("_size"):
            return super().__getattr__("any_workspace_size")
        return lambda *a: kb.OK


@pytest.fixture
def made(monkeypatch):
    """The tensors that the calls allocate, in order."""
    now, out = [CURRENT], []

    def set_stream(s):
        now[:] = [s]

    def empty(shape, dtype=F32, device=None):
        t = torch.zeros(shape, dtype=dtype).as_subclass(Noted)
        t.pool = now[0].cuda_stream
        out.append(t)
        return t

    class Torch:
        cuda = types.SimpleNamespace(Stream=Stream, set_stream=set_stream, current_stream=lambda *a: now[0])
        _C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: now[0].cuda_stream)

        def __getattr__(self, name):
            return empty if name == "empty" else getattr(torch, name)

    facade = Torch()
    monkeypatch.setattr(kb, "_torch", lambda: facade)
    monkeypatch.setattr(kb, "_device", lambda: 0)
    monkeypatch.setattr(kb, "lib", Quiet)
    for kept in ("_NORM_WS", "_ACT_WS"):
        monkeypatch.setattr(kb, kept, {})
    return out


def given(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Noted)


def weight(count=1, m=32, n=64):
    return kb.PackedWeight(given(4096, dtype=U8), count, m, n, 0, -8, False)


def layers():
    """name: (call of the stream, tensors it is given)."""
    x, y, rows, z = given(3, 64), given(3, 32), given(6, 64), given(3, 64)
    w, we, wi, wo = weight(), weight(2), weight(2, 16, 64), weight(2, 64, 8)
    place, wt, choice, offsets, dr = given(3, 2, dtype=I32), given(3, 2), given(3, 2, dtype=I32), given(3, dtype=I32), given(6, 32)
    b, v, router, mean, rstd = given(32), given(64), given(2, 64), given(3), given(3)
    return dict(
        linear=(lambda s: kb.bakron_linear(x, w, stream=s), (x, w.data)),
        linear_grad=(lambda s: kb.bakron_linear_grad(y, w, stream=s), (y, w.data)),
        linear_act=(lambda s: kb.bakron_linear_act(x, w, bias=b, act="silu", residual=y, want_pre=True, stream=s), (x, w.data, b, y)),
        act=(lambda s: kb.bakron_act(z, "silu", gated=True, stream=s), (z,)),
        act_grad=(lambda s: kb.bakron_act_grad(y, z, "silu", gated=True, want_bias_grad=True, stream=s), (y, z)),
        sort=(lambda s: kb.bakron_sort_tokens(choice, 4, stream=s), (choice,)),
        dispatch=(lambda s: kb.bakron_dispatch(x, place, wt, stream=s), (x, place, wt)),
        combine=(lambda s: kb.bakron_combine(rows, place, wt, stream=s), (rows, place, wt)),
        combine_grad=(lambda s: kb.bakron_combine_grad(x, rows, place, wt, stream=s), (x, rows, place, wt)),
        experts=(lambda s: kb.bakron_experts(rows, we, offsets, stream=s), (rows, we.data, offsets)),
        experts_grad=(lambda s: kb.bakron_experts_grad(dr, we, offsets, stream=s), (dr, we.data, offsets)),
        moe=(lambda s: kb.bakron_moe(x, router, wi, wo, 1, stream=s), (x, router, wi.data, wo.data)),
        norm=(lambda s: kb.bakron_layernorm(x, v, v, stream=s), (x, v)),
        norm_grad=(lambda s: kb.bakron_layernorm_grad(x, x, v, mean, rstd, stream=s), (x, v, mean, rstd)))


def solver():
    """Calls that wait for their stream: only what they allocate matters."""
    W, A, B, one, grid = given(32, 64), given(64, 64), given(32, 32), given(32), given(32, 1)
    codes = given(32, 64, dtype=I8)
    return dict(
        rowscale=lambda s: kb.bakron_rowscale(W, 7, stream=s),
        prepare=lambda s: kb.bakron_prepare(A, 0.0, B, 0.0, want_L=True, stream=s),
        quantize=lambda s: kb.bakron_quantize(W, A, B, one, -8, 7, want_preround=True, stream=s),
        params=lambda s: kb.bakron_grid_params(W, 4, stream=s),
        grid=lambda s: kb.bakron_quantize_grid(W, A, B, grid, grid, None, -8, 7, want_preround=True, stream=s),
        batch=lambda s: kb.bakron_quantize_batch([dict(W=W, UA=A, UB=B, scale=grid, qmin=-8, qmax=7)], stream=s),
        antidiag=lambda s: kb.bakron_quantize_antidiag(W, A, B, one, -8, 7, want_preround=True, stream=s),
        noalloc=lambda s: kb.bakron_quantize_noalloc(W, A, B, one, -8, 7, stream=s),
        factors=lambda s: kb.bakron_factors(W, W, stream=s),
        plan=lambda s: kb.bakron_plan_init(32, 64, stream=s),
        pack=lambda s: kb.bakron_pack(codes, grid, -8, 7, stream=s),
        unpack=lambda s: kb.bakron_unpack(weight(), stream=s),
        solver=lambda s: kb.Solver(32, 64, bits=4, opts=kb.Opts(), stream=s))


LAYERS = ["linear", "linear_grad", "linear_act", "act", "act_grad", "sort", "dispatch", "combine", "combine_grad", "experts",
          "experts_grad", "moe", "norm", "norm_grad"]
SOLVER = ["rowscale", "prepare", "quantize", "params", "grid", "batch", "antidiag", "noalloc", "factors", "plan", "pack", "unpack",
          "solver"]


@pytest.mark.parametrize("name", LAYERS + SOLVER)
def test_memory_of_the_calls_stream(made, name):
    call, inputs = layers()[name] if name in LAYERS else (solver()[name], ())
    call(SIDE)
    assert made, "nothing was allocated"
    for t in made:
        assert t.pool == SIDE.cuda_stream, "%s came from the current stream's memory" % (tuple(t.shape),)
        if t.dtype != U8 or name in ("plan", "pack"):       # no workspace
            assert CURRENT.cuda_stream in t.users, "the current stream may use what it is given back"
    for t in inputs:
        assert SIDE.cuda_stream in t.users, "an input may be let go while the call runs"


@pytest.mark.parametrize("name", ["linear", "experts", "norm", "dispatch", "act"])
def test_given_outputs_and_workspaces_stay_too(made, name):
    """What a caller passes for the outputs and the workspace may be let go as well."""
    ws, x, rows = given(4096, dtype=U8), given(3, 64), given(6, 64)
    w, offsets, place = weight(2), given(3, dtype=I32), given(3, 2, dtype=I32)
    call, more = dict(
        linear=(lambda **k: kb.bakron_linear(x, weight(), **k), dict(out=given(3, 32), workspace=ws)),
        experts=(lambda **k: kb.bakron_experts(rows, w, offsets, **k), dict(out=given(6, 32), workspace=ws)),
        norm=(lambda **k: kb.bakron_layernorm(x, want_stats=False, **k), dict(out=given(3, 64))),
        dispatch=(lambda **k: kb.bakron_dispatch(x, place, **k), dict(out=rows)),
        act=(lambda **k: kb.bakron_act(x, "silu", gated=True, **k), dict(out=given(3, 32))))[name]
    call(stream=SIDE, **more)
    assert not made
    for t in more.values():
        assert SIDE.cuda_stream in t.users


@pytest.mark.parametrize("stream", [None, CURRENT])
@pytest.mark.parametrize("name", LAYERS + SOLVER)
def test_the_current_stream(made, name, stream):
    call, inputs = layers()[name] if name in LAYERS else (solver()[name], ())
    call(stream)
    for t in made:
        assert t.pool == CURRENT.cuda_stream and not t.users
    for t in inputs:
        assert not t.users
