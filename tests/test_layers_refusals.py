"""fp32 arrays of the quantised layers' calls at addresses that are no multiple
of four are refused (no GPU: before any CUDA call)."""

import ctypes

import pytest

from test_layers_abi import ADDR, INVALID, kb, pack_bytes, packed  # noqa: F401


@pytest.mark.parametrize("bad", ["gamma", "beta", "mean", "rstd"])
def test_layernorm(kb, bad):  # noqa: F811
    a = dict(gamma=ADDR, beta=ADDR, mean=ADDR, rstd=ADDR)
    a[bad] += 2
    assert kb.lib().bakron_layernorm(ADDR, 4, 100, 1, a["gamma"], a["beta"], 0.1, ADDR, a["mean"], a["rstd"],
                                     None) == INVALID


@pytest.mark.parametrize("bad", ["gamma", "mean", "rstd", "dgamma", "dbeta"])
def test_layernorm_grad(kb, bad):  # noqa: F811
    a = dict(gamma=ADDR, mean=ADDR, rstd=ADDR, dgamma=ADDR, dbeta=ADDR)
    a[bad] += 2
    assert kb.lib().bakron_layernorm_grad(ADDR, ADDR, 4, 100, 1, a["gamma"], a["mean"], a["rstd"], ADDR, a["dgamma"],
                                          a["dbeta"], ADDR, 1 << 20, None) == INVALID


@pytest.mark.parametrize("scale,zero", [(ADDR + 2, None), (ADDR, ADDR + 1), (ADDR + 3, ADDR)])
def test_pack(kb, scale, zero):  # noqa: F811
    assert kb.lib().bakron_pack(ADDR, scale, zero, 1, 16, 128, 0, -8, 7, ADDR,
                                pack_bytes(1, 16, 128, 0, zero is not None), None) == INVALID


def test_unpack(kb):  # noqa: F811
    assert kb.lib().bakron_unpack(ctypes.byref(packed(kb)), ADDR + 2, None) == INVALID
