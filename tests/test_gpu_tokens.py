"""Tokens sorted by expert and back: bakron_sort_tokens, bakron_dispatch, bakron_combine and
bakron_combine_grad."""

import pytest

torch = pytest.importorskip("torch")

from _feedforward_helpers import check, places, random_choices, rounded
from _layer_helpers import U

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def _kb():
    from kronecker_factored_gptq_gb300 import bakron
    return bakron


def _randn(shape, dtype, seed):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 4), (5, 3, 7), (16, 2, 16), (31, 1, 33), (64, 32, 1000), (333, 6, 60),
                                   (1000, 4, 1024), (683, 3, 8), (5000, 8, 128), (70000, 2, 64), (40000, 8, 1)])
def test_sort(T, k, E, index):
    kb = _kb()
    choice = random_choices(T, k, E, T + k)
    if index == torch.int64 and T > 2:
        choice[1, 0] = (1 << 32) + E // 2        # no expert, though its low half is one
        choice[2, 0] = -(1 << 40)
    offsets, place = kb.bakron_sort_tokens(choice.to(index).cuda(), E)
    wo, wp = places(choice, E)
    assert offsets.dtype == place.dtype == torch.int32
    assert torch.equal(offsets.cpu(), wo) and torch.equal(place.cpu(), wp)


@pytest.mark.parametrize("T", [40, 4000])
def test_sort_of_one_expert_and_of_none(T):
    kb = _kb()
    for e in (3, -1, 9):
        choice = torch.full((T, 2), e, dtype=torch.int32)
        offsets, place = kb.bakron_sort_tokens(choice.cuda(), 9)
        wo, wp = places(choice, 9)
        assert torch.equal(offsets.cpu(), wo) and torch.equal(place.cpu(), wp)


def test_sort_of_no_tokens():
    kb = _kb()
    offsets, place = kb.bakron_sort_tokens(torch.empty((0, 2), dtype=torch.int64, device="cuda"), 5)
    assert (offsets == 0).all() and offsets.shape == (6,) and place.shape == (0, 2)


def test_sort_of_a_million_choices():
    kb = _kb()
    T, k, E = 131072, 8, 256
    choice = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    offsets, place = kb.bakron_sort_tokens(choice, E)
    flat = choice.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    want = torch.empty_like(order)
    want[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(place.reshape(-1).long(), want)
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)) and offsets[0] == 0


def _case(T, k, E, d, dtype, seed, lost=0.1):
    choice = random_choices(T, k, E, seed, lost)
    offsets, place = places(choice, E)
    g = torch.Generator().manual_seed(seed + 1)
    weight = torch.softmax(torch.randn((T, k), generator=g), 1)
    return place.cuda(), weight.cuda(), _randn((T, d), dtype, seed + 2), _randn((T * k, d), dtype, seed + 3)


SIZES = [(1, 1, 1, 1), (1, 8, 16, 4096), (2, 2, 4, 7), (5, 6, 8, 130), (37, 2, 8, 1111), (300, 4, 32, 64), (100, 5, 60, 1000),
         (64, 32, 64, 24), (33, 3, 4, 5000), (2000, 1, 4, 257), (9, 9, 9, 20000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,d", SIZES)
def test_dispatch_and_combine(T, k, E, d, dtype):
    kb = _kb()
    place, weight, x, rows = _case(T, k, E, d, dtype, T + d)
    live = place >= 0
    at = place[live].long()
    token = torch.nonzero(live)[:, 0]
    # out
    guard = torch.full((T * k, d), 7.0, dtype=dtype, device="cuda")
    want = guard.clone()
    want[at] = x[token]
    assert torch.equal(kb.bakron_dispatch(x, place, out=guard), want)
    out = kb.bakron_dispatch(x, place, weight, out=torch.full_like(guard, 7.0))
    ref = torch.full((T * k, d), 7.0, dtype=torch.float64, device="cuda")
    ref[at] = x.double()[token] * weight.double()[live][:, None]
    check(out, ref, rounded(U * ref.abs(), ref, dtype), "weighted rows")
    # and back
    for w in (None, weight):
        f = torch.ones_like(weight) if w is None else weight
        terms = torch.zeros((T, k, d), dtype=torch.float64, device="cuda")
        terms[live] = rows.double()[at] * f.double()[live][:, None]
        y = kb.bakron_combine(rows, place, w)
        ref = terms.sum(1)
        check(y, ref, rounded(U * (k + 1) * terms.abs().sum(1), ref, dtype), "y")
    none = (~live).all(1)
    assert (y[none] == 0).all()
    # gradients
    dy = _randn((T, d), dtype, 9)
    drows = torch.full((T * k, d), 7.0, dtype=dtype, device="cuda")
    drows, dweight = kb.bakron_combine_grad(dy, rows, place, weight, out=(drows, torch.full_like(weight, 7.0)))
    ref = torch.full((T * k, d), 7.0, dtype=torch.float64, device="cuda")
    ref[at] = dy.double()[token] * weight.double()[live][:, None]
    check(drows, ref, rounded(U * ref.abs(), ref, dtype), "drows")
    ref, mag = torch.zeros((T, k), dtype=torch.float64, device="cuda"), torch.zeros((T, k), dtype=torch.float64, device="cuda")
    ref[live] = (dy.double()[token] * rows.double()[at]).sum(1)
    mag[live] = (dy.double()[token] * rows.double()[at]).abs().sum(1)
    # a thread's columns one after the other (d / 32 at most), the lanes, the warps
    check(dweight, ref, U * (d / 32 + 8 + 5 + 8 + 1) * mag + 2.0 ** -149, "dweight")
    assert (dweight[~live] == 0).all()
    again = kb.bakron_combine_grad(dy, rows, place, weight, out=(drows.clone(), torch.empty_like(weight)))
    assert torch.equal(again[1], dweight), "two runs differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift,d", [(1, 64), (2, 64), (4, 64), (1, 33), (0, 34), (0, 36)])
def test_rows_at_odd_addresses(shift, d, dtype):
    """Rows that begin anywhere; what is beside them stays."""
    kb = _kb()
    T, k = 70, 3

    def odd(t):
        base = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device="cuda")
        v = base[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return base, v

    place, weight, x, rows = _case(T, k, 5, d, dtype, 3)
    want = kb.bakron_dispatch(x, place, out=torch.zeros_like(rows))
    base, out = odd(torch.zeros_like(rows))
    kb.bakron_dispatch(odd(x)[1], place, out=out)
    assert torch.equal(out, want) and (base[:shift] == 7).all() and (base[shift + out.numel():] == 7).all()
    y = kb.bakron_combine(rows, place, weight)
    base, out = odd(torch.zeros_like(x))
    kb.bakron_combine(odd(rows)[1], place, weight, out=out)
    assert torch.equal(out, y) and (base[:shift] == 7).all() and (base[shift + out.numel():] == 7).all()
    base, out = odd(torch.zeros_like(rows))
    got = kb.bakron_combine_grad(odd(x)[1], odd(rows)[1], place, weight, out=(out, torch.empty_like(weight)))
    ref = kb.bakron_dispatch(x, place, weight, out=torch.zeros_like(rows))
    assert torch.equal(got[0], ref) and (base[:shift] == 7).all() and (base[shift + out.numel():] == 7).all()
    dots = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    live = place >= 0
    a, b = x.double()[torch.nonzero(live)[:, 0]], rows.double()[place[live].long()]
    dots[live] = (a * b).sum(1)
    mag = torch.zeros_like(dots)
    mag[live] = (a * b).abs().sum(1)
    check(got[1], dots, U * (d / 32 + 22) * mag + 2.0 ** -149, "dweight")


def test_places_outside_the_rows_have_none():
    kb = _kb()
    T, k, d, R = 6, 2, 40, 5
    place = torch.tensor([[0, 5], [1, 6], [2, 1 << 30], [3, -2], [4, -(1 << 31)], [-1, 100]], dtype=torch.int32, device="cuda")
    x, rows, w = _randn((T, d), torch.float32, 1), _randn((R, d), torch.float32, 2), torch.full((T, k), 2.0, device="cuda")
    out = kb.bakron_dispatch(x, place, out=torch.zeros((R, d), device="cuda"))
    assert torch.equal(out, x[:5])
    y = kb.bakron_combine(rows, place, w)
    assert torch.equal(y[:5], 2 * rows) and (y[5] == 0).all()
    drows, dw = kb.bakron_combine_grad(x, rows, place, w)
    assert torch.equal(drows, 2 * x[:5]) and (dw[:, 1] == 0).all() and dw[5, 0] == 0
    # no rows at all
    none = torch.empty((0, d), device="cuda")
    assert (kb.bakron_combine(none, place, w) == 0).all()
    assert kb.bakron_dispatch(x, place, out=none).shape == (0, d)
    assert (kb.bakron_combine_grad(x, none, place, w)[1] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_what_no_choice_has_is_not_read(dtype):
    """NaN in rows without a choice and in weights of choices without a row."""
    kb = _kb()
    place, weight, x, rows = _case(50, 3, 6, 72, dtype, 4, lost=0.4)
    live = place >= 0
    y = kb.bakron_combine(rows, place, weight)
    g = kb.bakron_combine_grad(x, rows, place, weight, out=(torch.zeros_like(rows), torch.empty_like(weight)))
    used = torch.zeros(150, dtype=torch.bool, device="cuda")
    used[place[live].long()] = True
    rows2 = torch.where(used[:, None], rows, torch.full_like(rows, float("nan")))
    weight2 = torch.where(live, weight, torch.full_like(weight, float("nan")))
    assert torch.equal(kb.bakron_combine(rows2, place, weight2), y)
    g2 = kb.bakron_combine_grad(x, rows2, place, weight2, out=(torch.zeros_like(rows), torch.empty_like(weight)))
    assert torch.equal(g[0], g2[0]) and torch.equal(g[1], g2[1])


def test_nothing_to_do():
    kb = _kb()
    e, p, w = torch.empty((0, 8), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    rows = torch.ones((4, 8), device="cuda")
    assert torch.equal(kb.bakron_dispatch(e, p, out=rows.clone()), rows)
    assert kb.bakron_combine(rows, p).shape == (0, 8)
    drows, dw = kb.bakron_combine_grad(e, rows, p, w, out=(rows.clone(), w))
    assert torch.equal(drows, rows) and dw.shape == (0, 2)


def test_rows_beyond_32_bit_offsets():
    """More than 2^31 elements, and bytes, between the first row and the last."""
    kb = _kb()
    T, k, d, E = 70000, 8, 4096, 16
    choice = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    offsets, place = kb.bakron_sort_tokens(choice, E)
    x = torch.randn((T, d), dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    rows = kb.bakron_dispatch(x, place)
    assert rows.numel() > 1 << 31
    for t in (0, 1, 34567, T - 1):
        for j in range(k):
            assert torch.equal(rows[place[t, j].item()], x[t])
    w = torch.full((T, k), 0.125, device="cuda")
    y = kb.bakron_combine(rows, place, w)
    assert torch.equal(y, x)
    drows, dw = kb.bakron_combine_grad(x, rows, place, w)
    assert torch.equal(drows[place[T - 1].long()], (x[T - 1] * 0.125).expand(k, d))
    ref = x.double().square().sum(1)
    assert ((dw.double() - ref[:, None]).abs() <= U * (d / 32 + 22) * ref[:, None]).all()


@pytest.mark.parametrize("T", [16, 3000])
def test_in_a_graph_and_on_another_stream(T):
    """The whole way out and back, captured, with new choices on replay."""
    kb = _kb()
    k, E, d = 2, 8, 256
    choice = random_choices(T, k, E, 1).cuda()
    x = _randn((T, d), torch.bfloat16, 2)
    w = torch.full((T, k), 0.5, device="cuda")
    rows, y, dw = torch.zeros((T * k, d), dtype=torch.bfloat16, device="cuda"), torch.zeros_like(x), torch.zeros_like(w)
    sorted_ = (torch.zeros(E + 1, dtype=torch.int32, device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda"))
    drows = torch.zeros_like(rows)

    def way(stream=None):
        kb.bakron_sort_tokens(choice, E, out=sorted_, stream=stream)
        kb.bakron_dispatch(x, sorted_[1], out=rows, stream=stream)
        kb.bakron_combine(rows, sorted_[1], w, out=y, stream=stream)
        kb.bakron_combine_grad(x, rows, sorted_[1], w, out=(drows, dw), stream=stream)

    def right():
        wo, wp = places(choice.cpu(), E)
        assert torch.equal(sorted_[0].cpu(), wo) and torch.equal(sorted_[1].cpu(), wp)
        n = (sorted_[1] >= 0).sum(1, keepdim=True)
        assert torch.equal(y, (x.float() * 0.5 * n).to(torch.bfloat16))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    way(s)
    s.synchronize()
    right()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        way()
    for seed in (5, 6):
        choice.copy_(random_choices(T, k, E, seed))
        g.replay()
        torch.cuda.synchronize()
        right()
