"""Sizes and refusals of the quantised layers' entry points that need no GPU:
every refusal here returns before any CUDA call, so the addresses are never
read."""

import ctypes
import os

import pytest

ADDR = 1 << 20                       # aligned, never dereferenced
INVALID = 1


@pytest.fixture(scope="module")
def kb():
    from kronecker_factored_gptq_gb300 import bakron
    if not os.path.exists(bakron.LIB_PATH):
        from kronecker_factored_gptq_gb300 import build
        build.build()
    return bakron


def size(fn, *args):
    out = ctypes.c_size_t(0)
    st = fn(*args, ctypes.byref(out))
    return st, out.value


def pack_bytes(count, m, n, group, has_zero):
    """Header, codes, scales, zero points: the documented layout."""
    mp, np_ = -(-m // 16) * 16, -(-n // 128) * 128
    ng = 1 if group == 0 or group >= n else -(-n // group)
    b = 256 + count * mp * np_ // 2 + 4 * count * mp * ng + (count * mp * ng if has_zero else 0)
    return -(-b // 16) * 16


def packed(kb, m=64, n=256, group=64, count=1, **over):
    d = kb.Packed(count, m, n, group, 0, 0, ADDR, pack_bytes(count, m, n, group, False))
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("count,m,n,group,has_zero", [
    (1, 1, 1, 0, 0), (1, 16, 128, 128, 0), (3, 17, 129, 32, 1), (8, 4096, 14336, 128, 1), (2, 100, 1111, 96, 1)])
def test_pack_size(kb, count, m, n, group, has_zero):
    st, b = size(kb.lib().bakron_pack_size, count, m, n, group, has_zero)
    assert st == 0 and b == pack_bytes(count, m, n, group, has_zero)


@pytest.mark.parametrize("args", [
    (0, 16, 16, 0, 0), (1, 0, 16, 0, 0), (1, 16, 0, 0, 0), (1, 16, 128, 48, 0), (1, 16, 128, -32, 0),
    (1, (1 << 20) + 1, 16, 0, 0), (1, 16, (1 << 20) + 1, 0, 0), (1 << 20, 1 << 20, 1 << 20, 0, 0)])
def test_pack_size_refuses(kb, args):
    assert size(kb.lib().bakron_pack_size, *args)[0] == INVALID


def test_pack_refuses(kb):
    L = kb.lib()
    ok = dict(codes=ADDR, scale=ADDR, zero=None, count=1, m=16, n=128, group=0, qmin=-8, qmax=7, data=ADDR,
              bytes=pack_bytes(1, 16, 128, 0, False))
    for bad in (dict(codes=None), dict(scale=None), dict(data=None), dict(data=ADDR + 8), dict(qmin=7, qmax=-8),
                dict(qmin=-8, qmax=8), dict(qmin=-129, qmax=-120), dict(bytes=ok["bytes"] - 1), dict(group=48),
                dict(m=0)):
        a = dict(ok, **bad)
        assert L.bakron_pack(a["codes"], a["scale"], a["zero"], a["count"], a["m"], a["n"], a["group"], a["qmin"],
                             a["qmax"], a["data"], a["bytes"], None) == INVALID, bad


@pytest.mark.parametrize("T,dtype,grad,nbytes", [
    (0, 1, False, 0), (1, 1, False, 0), (16, 2, False, 0), (17, 1, False, 17 * 256 * 2), (300, 1, False, 300 * 256 * 2),
    (4, 0, False, 0), (100, 0, False, 3 * 100 * 256 * 2), (1, 1, True, 128 * 2), (5, 0, True, 3 * 5 * 128 * 2)])
def test_linear_workspace(kb, T, dtype, grad, nbytes):
    fn = kb.lib().bakron_linear_grad_workspace_size if grad else kb.lib().bakron_linear_workspace_size
    st, b = size(fn, ctypes.byref(packed(kb)), T, dtype)
    assert st == 0 and b == nbytes


@pytest.mark.parametrize("over", [dict(count=2, bytes=1 << 30), dict(data=None), dict(data=ADDR + 4), dict(bytes=512),
                                  dict(group=40), dict(qmin=-200), dict(m=0)])
@pytest.mark.parametrize("grad", [False, True])
def test_linear_refuses_the_weight(kb, over, grad):
    L = kb.lib()
    w = packed(kb, **over)
    fn = L.bakron_linear_grad if grad else L.bakron_linear
    assert fn(ADDR, 4, 1, ctypes.byref(w), ADDR, ADDR, 1 << 20, None) == INVALID


@pytest.mark.parametrize("grad", [False, True])
def test_linear_refuses_the_rest(kb, grad):
    L = kb.lib()
    w = packed(kb)
    r = ctypes.byref(w)
    fn = L.bakron_linear_grad if grad else L.bakron_linear
    for args in ((ADDR, -1, 1, r, ADDR, ADDR, 1 << 20), (ADDR, 4, 3, r, ADDR, ADDR, 1 << 20),
                 (ADDR, 4, 1, None, ADDR, ADDR, 1 << 20), (None, 4, 1, r, ADDR, ADDR, 1 << 20),
                 (ADDR, 4, 1, r, None, ADDR, 1 << 20), (ADDR + 1, 4, 1, r, ADDR, ADDR, 1 << 20),
                 (ADDR, 4, 0, r, ADDR + 2, ADDR, 1 << 20), (ADDR, 100, 1, r, ADDR, None, 0),
                 (ADDR, 100, 1, r, ADDR, ADDR + 16, 1 << 20), (ADDR, 100, 1, r, ADDR, ADDR, 100)):
        assert fn(*args, None) == INVALID, args
    assert fn(None, 0, 1, r, None, None, 0, None) == 0            # no tokens: nothing to do


def test_moe_refuses(kb):
    L = kb.lib()
    wi, wo = packed(kb, m=128, n=64, group=32, count=8), packed(kb, m=64, n=64, group=32, count=8)
    st, need = size(L.bakron_moe_workspace_size, ctypes.byref(wi), ctypes.byref(wo), 20, 2, 1)
    assert st == 0 and need > 0
    ok = dict(x=ADDR, T=20, dt=1, r=ADDR, wi=wi, wo=wo, k=2, y=ADDR, ws=ADDR, b=need)
    for bad in (dict(x=None), dict(r=None), dict(y=None), dict(ws=None), dict(ws=ADDR + 8), dict(b=need - 1),
                dict(T=-1), dict(dt=5), dict(k=0), dict(k=9), dict(k=17), dict(x=ADDR + 1),
                dict(wi=packed(kb, m=130, n=64, group=32, count=8)), dict(wi=packed(kb, m=128, n=64, group=32, count=4)),
                dict(wo=packed(kb, m=80, n=64, group=32, count=8))):
        a = dict(ok, **bad)
        assert L.bakron_moe(a["x"], a["T"], a["dt"], a["r"], ctypes.byref(a["wi"]), ctypes.byref(a["wo"]), a["k"], 1,
                            a["y"], a["ws"], a["b"], None) == INVALID, bad
    assert L.bakron_moe(None, 0, 1, None, ctypes.byref(wi), ctypes.byref(wo), 2, 1, None, None, 0, None) == 0


def test_layernorm_refuses(kb):
    L = kb.lib()
    for T, d, dt, x, y, eps in ((-1, 8, 0, ADDR, ADDR, 0.1), (4, 0, 0, ADDR, ADDR, 0.1), (4, (1 << 20) + 1, 0, ADDR, ADDR, 0.1),
                                (4, 8, 3, ADDR, ADDR, 0.1), (4, 8, 0, None, ADDR, 0.1), (4, 8, 0, ADDR, None, 0.1),
                                (4, 8, 0, ADDR + 2, ADDR, 0.1), (4, 8, 1, ADDR, ADDR + 1, 0.1), (4, 8, 0, ADDR, ADDR, -1.0),
                                (4, 8, 0, ADDR, ADDR, float("nan"))):
        assert L.bakron_layernorm(x, T, d, dt, None, None, eps, y, None, None, None) == INVALID
    assert L.bakron_layernorm(None, 0, 8, 0, None, None, 0.0, None, None, None, None) == 0
    st, need = size(L.bakron_layernorm_grad_workspace_size, 4, 100)
    assert st == 0 and need >= 2 * 100 * 4
    ok = dict(dy=ADDR, x=ADDR, T=4, d=100, dt=0, mean=ADDR, rstd=ADDR, dx=ADDR, dg=ADDR, db=ADDR, ws=ADDR, b=need)
    for bad in (dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(dg=None), dict(db=None),
                dict(ws=None), dict(b=need - 1), dict(ws=ADDR + 4), dict(T=-1), dict(d=0), dict(dt=9), dict(dx=ADDR + 1)):
        a = dict(ok, **bad)
        assert L.bakron_layernorm_grad(a["dy"], a["x"], a["T"], a["d"], a["dt"], None, a["mean"], a["rstd"], a["dx"],
                                       a["dg"], a["db"], a["ws"], a["b"], None) == INVALID, bad
