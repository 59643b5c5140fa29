"""Sizes and refusals of the feed-forward calls that need no GPU: every refusal
returns before any CUDA call, so the addresses are never read."""

import ctypes

import pytest

from test_layers_abi import ADDR, INVALID, kb, pack_bytes, packed, size  # noqa: F401

BIG = 1 << 30


def refused(fn, ok, bad, *names):
    for b in bad:
        a = dict(ok, **b)
        assert fn(*(a[n] for n in names)) == INVALID, b


def test_linear_act(kb):  # noqa: F811
    r = ctypes.byref(packed(kb))
    two = packed(kb, count=2, bytes=BIG)
    ok = dict(x=ADDR, T=100, dt=1, w=r, bias=ADDR, act=4, res=ADDR, y=ADDR, pre=ADDR, ws=ADDR, b=1 << 20, s=None)
    refused(kb.lib().bakron_linear_act, ok, [
        dict(x=None), dict(y=None), dict(T=-1), dict(T=(1 << 28) + 1), dict(dt=3), dict(dt=-1), dict(w=None),
        dict(w=ctypes.byref(two)), dict(act=-1), dict(act=5), dict(bias=ADDR + 2), dict(res=ADDR + 1), dict(pre=ADDR + 1),
        dict(dt=0, res=ADDR + 2), dict(dt=0, pre=ADDR + 2), dict(x=ADDR + 1), dict(y=ADDR + 1), dict(ws=None),
        dict(ws=ADDR + 16), dict(b=100)], *ok)
    assert kb.lib().bakron_linear_act(None, 0, 1, r, None, 0, None, None, None, None, 0, None) == 0


def test_act(kb):  # noqa: F811
    L = kb.lib()
    ok = dict(z=ADDR, T=4, m=10, dt=1, act=4, gated=1, y=ADDR, s=None)
    refused(L.bakron_act, ok, [
        dict(z=None), dict(y=None), dict(T=-1), dict(T=(1 << 28) + 1), dict(m=0), dict(m=(1 << 20) + 1), dict(dt=3), dict(act=5),
        dict(act=-1), dict(gated=2), dict(z=ADDR + 1), dict(dt=0, y=ADDR + 2)], *ok)
    assert L.bakron_act(None, 0, 10, 1, 4, 0, None, None) == 0
    ok = dict(dy=ADDR, z=ADDR, T=4000, m=64, dt=1, act=4, gated=0, dz=ADDR, db=ADDR, ws=ADDR, b=1 << 24, s=None)
    st, need = size(L.bakron_act_grad_workspace_size, 4000, 64)
    assert st == 0 and need > 0 and need % (64 * 4) == 0
    refused(L.bakron_act_grad, ok, [
        dict(dy=None), dict(z=None), dict(dz=None), dict(T=-1), dict(m=0), dict(dt=9), dict(act=7), dict(gated=-1),
        dict(db=ADDR + 2), dict(dz=ADDR + 1), dict(dy=ADDR + 1), dict(z=ADDR + 1), dict(ws=None), dict(ws=ADDR + 64),
        dict(b=need - 1)], *ok)
    assert L.bakron_act_grad(None, None, 0, 64, 1, 4, 0, None, None, None, 0, None) == 0


@pytest.mark.parametrize("T,columns", [(0, 1), (1, 1), (4, 100000), (37, 1111), (100000, 8), (100000, 64), (8192, 28672)])
def test_act_grad_workspace(kb, T, columns):  # noqa: F811
    """What one call needs serves every call with fewer rows."""
    st, need = size(kb.lib().bakron_act_grad_workspace_size, T, columns)
    assert st == 0
    for t in (0, 1, T // 7, T // 2, max(0, T - 1)):
        st, less = size(kb.lib().bakron_act_grad_workspace_size, min(t, T), columns)
        assert st == 0 and less <= need
    for bad in ((-1, 8), ((1 << 28) + 1, 8), (8, 0), (8, (1 << 21) + 1)):
        assert size(kb.lib().bakron_act_grad_workspace_size, *bad)[0] == INVALID


def test_sort_tokens(kb):  # noqa: F811
    ok = dict(c=ADDR, bytes=8, T=10, k=2, E=8, o=ADDR, p=ADDR, s=None)
    refused(kb.lib().bakron_sort_tokens, ok, [
        dict(c=None), dict(bytes=2), dict(bytes=0), dict(T=-1), dict(k=0), dict(k=33), dict(T=1 << 28), dict(E=0), dict(E=1025),
        dict(o=None), dict(p=None), dict(o=ADDR + 2), dict(p=ADDR + 1), dict(c=ADDR + 4), dict(bytes=4, c=ADDR + 2)], *ok)


def test_rows(kb):  # noqa: F811
    L = kb.lib()
    ok = dict(x=ADDR, T=10, d=64, dt=1, p=ADDR, k=2, w=ADDR, rows=ADDR, R=20, s=None)
    bad = [dict(x=None), dict(T=-1), dict(d=0), dict(d=(1 << 20) + 1), dict(dt=3), dict(p=None), dict(k=0), dict(k=33),
           dict(T=1 << 28), dict(R=-1), dict(R=(1 << 28) + 1), dict(rows=None), dict(x=ADDR + 1), dict(rows=ADDR + 1),
           dict(p=ADDR + 2), dict(w=ADDR + 2), dict(dt=0, x=ADDR + 2), dict(dt=0, rows=ADDR + 2)]
    refused(L.bakron_dispatch, ok, bad, *ok)
    refused(L.bakron_combine, ok, bad, "rows", "R", "d", "dt", "p", "T", "k", "w", "x", "s")
    ok = dict(ok, drows=ADDR, dw=ADDR)
    refused(L.bakron_combine_grad, ok, bad + [dict(w=None), dict(drows=None), dict(dw=None), dict(dw=ADDR + 2), dict(drows=ADDR + 1)],
            "x", "rows", "R", "d", "dt", "p", "T", "k", "w", "drows", "dw", "s")
    assert L.bakron_dispatch(None, 0, 64, 1, None, 2, None, None, 0, None) == 0
    assert L.bakron_dispatch(ADDR, 5, 64, 1, ADDR, 2, None, None, 0, None) == 0      # no rows: nothing to write
    assert L.bakron_combine(ADDR, 20, 64, 1, None, 0, 2, None, None, None) == 0
    assert L.bakron_combine_grad(None, ADDR, 20, 64, 1, None, 0, 2, None, None, None, None) == 0


@pytest.mark.parametrize("grad", [False, True])
def test_experts(kb, grad):  # noqa: F811
    L = kb.lib()
    fn = L.bakron_experts_grad if grad else L.bakron_experts
    w = packed(kb, count=4, bytes=BIG)
    r = ctypes.byref(w)
    st, need = size(L.bakron_experts_workspace_size, r, 100, 1, int(grad))
    assert st == 0 and need >= 100 * (128 if grad else 256) * 2
    for R in (0, 1, 50, 99):
        st, less = size(L.bakron_experts_workspace_size, r, R, 1, int(grad))
        assert st == 0 and less <= need
    many, odd = packed(kb, count=1025, bytes=BIG), packed(kb, count=4, bytes=BIG, group=40)
    ok = dict(x=ADDR, R=100, dt=1, w=r, o=ADDR, y=ADDR, ws=ADDR, b=need, s=None)
    refused(fn, ok, [
        dict(x=None), dict(y=None), dict(o=None), dict(o=ADDR + 2), dict(R=-1), dict(R=(1 << 28) + 1), dict(dt=5), dict(w=None),
        dict(w=ctypes.byref(many)), dict(w=ctypes.byref(odd)), dict(x=ADDR + 1), dict(dt=0, y=ADDR + 2), dict(ws=None),
        dict(ws=ADDR + 8), dict(b=need - 1)], *ok)
    assert fn(None, 0, 1, r, None, None, None, 0, None) == 0
    for bad in ((None, 100, 1, 0), (r, -1, 1, 0), (r, 100, 3, 0), (r, 100, 1, 2), (ctypes.byref(many), 100, 1, 0)):
        assert size(L.bakron_experts_workspace_size, *bad)[0] == INVALID


def test_binding_names_the_activations(kb):  # noqa: F811
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "bakron.h")).read()
    found = {n.lower(): int(v) for n, v in re.findall(r"BAKRON_ACT_([A-Z_]+) = (\d+)", text)}
    assert found == kb.ACTIVATIONS
