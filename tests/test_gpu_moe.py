"""bakron_moe against the plain 64-bit form."""

import pytest

torch = pytest.importorskip("torch")

from _layer_helpers import HALF_ULP, TINY, U, product_depth, random_weight, value

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _layer(E, d, f, group, asym, seed):
    ci, si, zi, qmin, qmax = random_weight((E, 2 * f, d), group, asym, seed)
    co, so, zo, _, _ = random_weight((E, d, f), group, asym, seed + 1)
    # values of about 1 / sqrt(length), so that h and y are of the order of x
    si, so = si * 25 / d ** 0.5, so * 25 / f ** 0.5
    kb = _kb()
    w_in = kb.bakron_pack(ci, si, qmin, qmax, zero=zi, group=group)
    w_out = kb.bakron_pack(co, so, qmin, qmax, zero=zo, group=group)
    return w_in, w_out, value(ci, si, zi, group), value(co, so, zo, group)


def _tokens(T, E, d, dtype, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn((T, d), generator=g).to(dtype).cuda()
    r = (torch.randn((E, d), generator=g) / d ** 0.5).to(dtype).cuda()
    return x, r


def reference(x, r, Vi, Vo, k, renormalize):
    """(y, bound on the fp32 error of y before its rounding, ids): one token
    and one of its experts at a time.  The bound adds, to first order, what the
    logits' sums, the two products and silu may be off in fp32."""
    x, r = x.double(), r.double()
    T, d = x.shape
    f = Vo.shape[2]
    logits = x @ r.T
    e_logit = 2 * U * (d / 8 + 16) * (x.abs() @ r.abs().T)
    y, err, ids = torch.zeros_like(x), torch.zeros_like(x), []
    for t in range(T):
        l = logits[t].tolist()
        best = sorted(range(len(l)), key=lambda e: (-l[e], e))
        ids.append(best[:k])
        p = torch.softmax(logits[t], 0)
        q = p[best[:k]]
        if renormalize:
            q = q / q.sum()
        eq = 2 * e_logit[t].max() + 8 * U * (1 + len(l) / 32)     # relative error of a weight
        for w, e in zip(q, best[:k]):
            gu, mag = Vi[e] @ x[t], Vi[e].abs() @ x[t].abs()
            egu = 2 * U * product_depth(d) * mag
            g, u = gu[:f], gu[f:]
            s = g * torch.sigmoid(g)
            h = s * u
            # |silu'| <= 1.1; silu itself to a few roundings
            eh = 1.1 * egu[:f] * u.abs() + (s.abs() + 1.1 * egu[:f]) * egu[f:] + 8 * U * h.abs()
            eh = eh + 2.0 ** -16 * h.abs()                        # two bf16 terms of h
            y[t] += w * (Vo[e] @ h)
            err[t] += w * (Vo[e].abs() @ (eh + (eq + 2 * U * (product_depth(f) + 2 * k)) * h.abs()))
    return y, err, ids


def check(y, x, r, Vi, Vo, k, renormalize, dtype):
    ref, err, ids = reference(x, r, Vi, Vo, k, renormalize)
    tol = 1.01 * err + HALF_ULP[dtype] * (ref.abs() + err) + TINY[dtype]
    assert torch.isfinite(y).all()
    worst = ((y.double() - ref).abs() / tol).max().item()
    assert worst <= 1.0, "error %.3g times the bound" % worst
    return ids


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k,d,f,group,asym,renormalize", [
    (1, 4, 1, 128, 64, 0, False, True), (1, 8, 2, 256, 128, 128, True, False), (1, 32, 4, 300, 100, 32, True, True),
    (2, 3, 3, 65, 33, 0, False, True), (5, 16, 2, 192, 88, 64, False, False), (8, 8, 2, 512, 256, 128, False, True),
    (9, 60, 6, 129, 40, 96, True, True), (16, 8, 2, 1024, 200, 128, False, True), (17, 4, 2, 256, 300, 32, False, True),
    (32, 8, 8, 136, 72, 64, True, False), (33, 16, 4, 128, 128, 0, False, True), (70, 5, 2, 100, 50, 32, True, True),
    (3, 1, 1, 64, 1, 0, False, True), (4, 300, 16, 72, 24, 0, True, False), (1, 2, 1, 1, 1, 0, False, True)])
def test_moe(T, E, k, d, f, group, asym, renormalize, dtype):
    kb = _kb()
    w_in, w_out, Vi, Vo = _layer(E, d, f, group, asym, T + E + d)
    x, r = _tokens(T, E, d, dtype, f)
    y = kb.bakron_moe(x, r, w_in, w_out, k, renormalize=renormalize)
    assert y.shape == (T, d) and y.dtype == dtype
    check(y, x, r, Vi, Vo, k, renormalize, dtype)
    assert torch.equal(y, kb.bakron_moe(x, r, w_in, w_out, k, renormalize=renormalize)), "two runs differ"


def test_ties_go_to_the_lowest_index():
    """Experts 1, 2 and 5 share a router row: with equal logits the first ones
    are chosen."""
    kb = _kb()
    E, d, f = 8, 128, 64
    w_in, w_out, Vi, Vo = _layer(E, d, f, 0, False, 3)
    x, r = _tokens(6, E, d, torch.float32, 4)
    r[2] = r[1]
    r[5] = r[1]
    y = kb.bakron_moe(x, r, w_in, w_out, 2)
    ids = check(y, x, r, Vi, Vo, 2, True, torch.float32)
    assert any(i[:2] == [1, 2] for i in ids) or any(1 in i for i in ids)
    z = torch.zeros_like(r)      # every logit 0: experts 0 and 1, weights a half
    y = kb.bakron_moe(x, z, w_in, w_out, 2)
    assert check(y, x, z, Vi, Vo, 2, True, torch.float32) == [[0, 1]] * 6


def test_one_expert_takes_all_and_far_logits():
    kb = _kb()
    E, d, f = 6, 128, 96
    w_in, w_out, Vi, Vo = _layer(E, d, f, 32, True, 5)
    x, r = _tokens(20, E, d, torch.float32, 6)
    x = x.abs() + 0.1
    r = r * 0 - 5.0
    r[4] = 5.0                   # logits of about +-600: the others' weights vanish
    y = kb.bakron_moe(x, r, w_in, w_out, 1)
    assert check(y, x, r, Vi, Vo, 1, True, torch.float32) == [[4]] * 20
    y = kb.bakron_moe(x, r, w_in, w_out, 2, renormalize=False)
    check(y, x, r, Vi, Vo, 2, False, torch.float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_stays_in_its_row(dtype):
    kb = _kb()
    w_in, w_out, Vi, Vo = _layer(8, 128, 64, 0, False, 7)
    x, r = _tokens(9, 8, 128, dtype, 8)
    x[4, 17] = float("nan")
    y = kb.bakron_moe(x, r, w_in, w_out, 2)
    assert torch.isnan(y[4]).all()
    keep = [t for t in range(9) if t != 4]
    check(y[keep], x[keep], r, Vi, Vo, 2, True, dtype)


def test_nan_in_the_router_alone():
    """A router row of NaN: every logit of that expert is NaN, so every row is."""
    kb = _kb()
    w_in, w_out, _, _ = _layer(4, 64, 32, 0, False, 9)
    x, r = _tokens(3, 4, 64, torch.float32, 10)
    r[3] = float("nan")
    for renormalize in (True, False):
        assert torch.isnan(kb.bakron_moe(x, r, w_in, w_out, 2, renormalize=renormalize)).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_unaligned_rows(dtype):
    kb = _kb()
    T, E, d, f = 6, 8, 256, 64
    w_in, w_out, Vi, Vo = _layer(E, d, f, 64, True, 11)
    x, r = _tokens(T, E, d, dtype, 12)

    def off(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.reshape(-1)
        return b[1:].view(t.shape)

    x, r = off(x), off(r)
    obase = torch.full((T * d + 2,), 7.0, dtype=dtype, device="cuda")
    out = obase[1:-1].view(T, d)
    kb.bakron_moe(x, r, w_in, w_out, 2, out=out)
    check(out, x, r, Vi, Vo, 2, True, dtype)
    assert obase[0] == 7.0 and obase[-1] == 7.0


def test_in_a_graph_and_on_another_stream():
    kb = _kb()
    w_in, w_out, _, _ = _layer(16, 256, 128, 128, False, 13)
    x, r = _tokens(4, 16, 256, torch.bfloat16, 14)
    want = kb.bakron_moe(x, r, w_in, w_out, 4)
    out, ws = torch.empty_like(want), kb.moe_workspace(w_in, w_out, 4, 4, x.dtype)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kb.bakron_moe(x, r, w_in, w_out, 4, out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    late = torch.zeros_like(x)
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)
        late.copy_(x)
    kb.bakron_moe(late, r, w_in, w_out, 4, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_refusals():
    kb = _kb()
    w_in, w_out, _, _ = _layer(4, 64, 32, 0, False, 15)
    other, _, _, _ = _layer(4, 64, 48, 0, False, 16)
    x, r = _tokens(2, 4, 64, torch.float32, 17)
    assert kb.bakron_moe(x[:0], r, w_in, w_out, 2).shape == (0, 64)
    with pytest.raises(ValueError):
        kb.bakron_moe(x, r, other, w_out, 2)
    with pytest.raises(ValueError):
        kb.bakron_moe(x, r.bfloat16(), w_in, w_out, 2)
    with pytest.raises(ValueError):
        kb.bakron_moe(x, r[:3], w_in, w_out, 2)
    with pytest.raises(ValueError):
        kb.bakron_moe(x, r, w_in, w_out, 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for k in (0, 5):
        with pytest.raises(kb.BakronError) as e:
            kb.bakron_moe(x, r, w_in, w_out, k)
        assert e.value.status == 1
