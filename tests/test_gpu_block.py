"""The quantised layers' calls together: the example that quantises a block,
tunes its norm through the packed layer and answers single tokens."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("tune_quantized_block",
                                                  os.path.join(ROOT, "examples", "tune_quantized_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype,sizes", [
    (torch.bfloat16, dict(tokens=300, d=200, m=136, experts=4, f=72, group=64)),
    (torch.float32, dict(tokens=130, d=129, m=65, experts=3, f=40, group=32))])
def test_example(dtype, sizes):
    losses, sides, answers, together = _example().run(dtype=dtype, steps=4, **sizes)
    assert all(b <= a * 1.01 for a, b in zip(losses, losses[1:])) and losses[-1] < losses[0]
    assert 0 < sides[1] < sides[0]
    # each is rounded once to its type, from fp32 sums in another order
    scale = together.float().abs().max().item()
    tol = 2 * torch.finfo(dtype).eps * together.float().abs() + 1e-3 * scale
    assert ((answers.float() - together.float()).abs() <= tol).all()
