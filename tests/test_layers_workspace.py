"""Workspace of the linear layer's gradient for long sums (no GPU): 16-bit
chains beyond 4096 rows (fp16) or 32768 (bf16) take N x 128 floats per block
behind the planes of dY."""

import ctypes
import os

import pytest

ADDR = 1 << 20


@pytest.fixture(scope="module")
def kb():
    from kronecker_factored_gptq_gb300 import bakron
    if not os.path.exists(bakron.LIB_PATH):
        from kronecker_factored_gptq_gb300 import build
        build.build()
    return bakron


@pytest.mark.parametrize("T,m,dtype,more", [
    (40, 4096, 2, False), (40, 4097, 2, True), (1000, 5000, 2, True), (40, 32768, 1, False), (7, 32769, 1, True),
    (40, 40000, 0, False), (0, 5000, 2, False)])
def test_gradient_workspace(kb, T, m, dtype, more):
    d = kb.Packed(1, m, 128, 0, 0, 0, ADDR, 1 << 30)
    b = ctypes.c_size_t(0)
    assert kb.lib().bakron_linear_grad_workspace_size(ctypes.byref(d), T, dtype, ctypes.byref(b)) == 0
    want = (3 if dtype == 0 else 1) * T * (-(-m // 128) * 128) * 2
    if more:
        want = -(-want // 256) * 256 + kb.sm_count() * min(256, -(-T // 32) * 32) * 128 * 4
    assert b.value == want
    # what one call needs serves every call with fewer tokens
    for t in range(1, T, 37):
        s = ctypes.c_size_t(0)
        assert kb.lib().bakron_linear_grad_workspace_size(ctypes.byref(d), t, dtype, ctypes.byref(s)) == 0
        assert s.value <= b.value
