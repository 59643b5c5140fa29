"""The quantised layers' Python calls launch on the current device: tensors,
weights, workspaces and streams of another one are refused, and what is kept
per size is kept per device.  No GPU: tensors that say where they are."""

import pytest

torch = pytest.importorskip("torch")

from kronecker_factored_gptq_gb300 import bakron as kb


class Placed(torch.Tensor):
    """A CPU tensor that answers as one on CUDA device ``index``."""

    index = 0
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index


class Placed1(Placed):
    index = 1


def on(index, *shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(Placed1 if index else Placed)


class Called(Exception):
    pass


class Library:
    """Stands for the library: sizes are (some function of) the device, and a
    call that reaches it says so."""

    def __getattr__(self, name):
        if name == "bakron_layernorm_grad_workspace_size":
            def size(T, d, out):
                out._obj.value = 1000 * (1 + kb._device())
                return kb.OK
            return size
        if name.endswith(("_workspace_size", "pack_size")):
            def size(*a):
                a[-1]._obj.value = 64
                return kb.OK
            return size

        def call(*a):
            raise Called(name)
        return call


class Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device_index = index


@pytest.fixture
def device(monkeypatch):
    """The current device, as a list of one number."""
    now = [0]
    monkeypatch.setattr(kb, "_torch", lambda: torch)
    monkeypatch.setattr(kb, "_device", lambda: now[0], raising=False)
    monkeypatch.setattr(kb, "lib", Library)
    monkeypatch.setattr(kb, "_NORM_WS", {})
    return now


def weight(index, count=1, m=32, n=64):
    return kb.PackedWeight(on(index, 4096, dtype=torch.uint8), count, m, n, 0, -8, False)


def calls(index, workspace=None, stream=Stream(0)):
    """Each call with everything on one device."""
    x, y = on(index, 3, 64), on(index, 3, 32)
    w, wi, wo = weight(index), weight(index, 2, 16, 64), weight(index, 2, 64, 8)
    keep = dict(workspace=workspace, stream=stream)
    return [lambda: kb.bakron_linear(x, w, out=y, **keep), lambda: kb.bakron_linear_grad(y, w, out=x, **keep),
            lambda: kb.bakron_moe(x, on(index, 2, 64), wi, wo, 1, out=on(index, 3, 64), **keep),
            lambda: kb.bakron_layernorm(x, out=on(index, 3, 64), want_stats=False, stream=stream),
            lambda: kb.bakron_layernorm_grad(x, x, None, on(index, 3), on(index, 3), want_weight_grads=False,
                                             out=on(index, 3, 64), stream=stream)]


def norm_grad(index, workspace):
    x = on(index, 3, 64)
    kb.bakron_layernorm_grad(x, x, None, on(index, 3), on(index, 3), out=on(index, 3, 64), workspace=workspace,
                             stream=Stream(0))


@pytest.mark.parametrize("which", range(5))
def test_tensors_of_another_device(device, which):
    ws = on(0, 4096, dtype=torch.uint8)
    with pytest.raises(Called):
        calls(0, ws)[which]()
    with pytest.raises(ValueError, match="current device"):
        calls(1, on(1, 4096, dtype=torch.uint8))[which]()
    device[0] = 1
    with pytest.raises(ValueError, match="current device"):
        calls(0, ws)[which]()


@pytest.mark.parametrize("which", range(5))
def test_a_stream_of_another_device(device, which):
    with pytest.raises(ValueError, match="stream"):
        calls(0, on(0, 4096, dtype=torch.uint8), Stream(1))[which]()


@pytest.mark.parametrize("which", range(3))
def test_workspaces(device, which):
    for bad in (torch.zeros(4096, dtype=torch.uint8), on(1, 4096, dtype=torch.uint8), on(0, 63, dtype=torch.uint8),
                on(0, 4096, dtype=torch.uint8)[::2], on(0, 256, 4)[:, :3]):
        with pytest.raises(ValueError, match="workspace"):
            calls(0, bad)[which]()
        if which == 0:
            with pytest.raises(ValueError, match="workspace"):
                norm_grad(0, bad if bad.numel() != 63 else on(0, 999, dtype=torch.uint8))


def test_packing_and_unpacking(device):
    codes, scale = on(1, 16, 32, dtype=torch.int8), on(1, 16, 1)
    with pytest.raises(ValueError, match="current device"):
        kb.bakron_pack(codes, scale, -8, 7)
    with pytest.raises(ValueError, match="current device"):
        kb.bakron_unpack(weight(1))
    with pytest.raises(ValueError, match="scale is on cuda:1"):
        kb.bakron_pack(on(0, 16, 32, dtype=torch.int8), scale, -8, 7)


def test_norm_workspace_sizes_are_kept_per_device(device):
    assert kb.layernorm_grad_workspace_size(5, 64) == 1000
    device[0] = 1
    assert kb.layernorm_grad_workspace_size(5, 64) == 2000
    device[0] = 0
    assert kb.layernorm_grad_workspace_size(5, 64) == 1000


def test_workspace_sizes_are_asked_on_the_weights_device(device):
    w, wi, wo = weight(1), weight(1, 2, 16, 64), weight(1, 2, 64, 8)
    for ask in (lambda: kb.linear_workspace_size(w, 5, torch.float32),
                lambda: kb.linear_workspace_size(w, 5, torch.float32, grad=True),
                lambda: kb.moe_workspace_size(wi, wo, 5, 1, torch.float32)):
        with pytest.raises(ValueError, match="current device"):
            ask()
        device[0] = 1
        assert ask() == 64
        device[0] = 0
