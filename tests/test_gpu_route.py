"""GPU parity of the router against the FP64 oracle.

Choices, counts and the places of the gates are equal.  Tolerances of the
values: a weight is scale s / sum; exp of a difference |d| <= 32 is off by
(32 + 2) u of itself from the difference's rounding and the function, a sum
of at most 512 by (16 + 9 + 34) u, the divisions and the scale by 4 u: 160 u
in all of |w| (the sums of a softmax enter numerator and denominator).  A
logit's gradient is a sum of products of such weights with d: 320 u of the sum
of magnitudes |w| (|d| + sum |d w| / scale).
"""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -24
LOW = float(np.finfo(np.float32).min)


def C():
    from equivariant_mlip_clebsch_b200 import cgtp
    return cgtp


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def T(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def back(kw):
    return {k: v for k, v in kw.items() if k in ("score", "renormalise", "scale")}


def compare(kw, l, bias, dev, seed=1):
    n, E = l.shape
    r = C().Router(E, **kw)
    ld_ = T(l, dev)
    b_ = None if bias is None else T(bias, dev)
    ids, w, gates, counts = r.forward(ld_, b_)
    oi, ow, og, oc, _ = O.route_forward(l, bias, **kw)
    assert np.array_equal(ids.cpu().numpy(), oi)
    assert np.array_equal(counts.cpu().numpy(), oc)
    wn = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(wn - ow) <= 160 * U * ow + 1e-38)
    # the gates hold exactly the weights
    ref = np.zeros((E + 1, n), np.float32)
    ref[np.where(oi < 0, E, oi), np.arange(n)[:, None]] = w.cpu().numpy()
    assert np.array_equal(gates.cpu().numpy(), ref[:E])
    rng = np.random.default_rng(seed)
    gw, gg = rng.standard_normal((n, kw["k"])).astype(np.float32), rng.standard_normal((E, n)).astype(np.float32)
    for a, c in ((gw, gg), (None, gg), (gw, None)):
        d = r.backward(ld_, ids, None if a is None else T(a, dev), None if c is None else T(c, dev))
        ref = O.route_backward(l, oi, a, c, **back(kw))
        held = oi >= 0
        dd = np.where(held, (0 if a is None else np.abs(a)) +
                      (0 if c is None else np.abs(c[np.maximum(oi, 0), np.arange(n)[:, None]])), 0.0)
        dot = (dd * ow).sum(1, keepdims=True) / kw.get("scale", 1.0)
        mag = np.zeros((n, E + 1))
        np.put_along_axis(mag, np.where(held, oi, E), ow * (dd + (dot if kw.get("renormalise", True) else 0)), 1)
        mag = mag[:, :E]
        if kw.get("score", "softmax") == "softmax" and not kw.get("renormalise", True):
            s = O.route_forward(l, None, kw["k"])[4]
            mag = mag + s * kw.get("scale", 1.0) * dot
        err = np.abs(d.cpu().numpy().astype(np.float64) - ref)
        assert np.all(err <= 320 * U * mag + 1e-37), float((err - 320 * U * mag).max())
    return r, ids, w, gates, counts


ROUTES = [(4, dict(k=1, score="softmax", renormalise=False)), (16, dict(k=2, score="softmax", renormalise=False)),
          (64, dict(k=8, score="sigmoid", n_groups=8, top_groups=4, scale=2.5)), (5, dict(k=5, score="sigmoid")),
          (1, dict(k=1)), (33, dict(k=3, score="softmax", n_groups=3, top_groups=2, group_best=1)),
          (256, dict(k=8, score="sigmoid", n_groups=8, top_groups=3, renormalise=False)),
          (257, dict(k=6, score="softmax")), (512, dict(k=32, score="softmax", renormalise=False, scale=0.5)),
          (63, dict(k=9, score="sigmoid", n_groups=7, top_groups=7)), (12, dict(k=4, n_groups=12, top_groups=5)),
          (130, dict(k=8, score="softmax", n_groups=2, top_groups=1, renormalise=False)),
          (64, dict(k=16, n_groups=32, top_groups=9, group_best=1)), (8, dict(k=8, score="sigmoid", renormalise=False))]


@pytest.mark.parametrize("E,kw", ROUTES)
@pytest.mark.parametrize("n", [1, 3, 37, 300, 1501])
@pytest.mark.parametrize("bias", [False, True])
def test_route_matches_the_oracle(E, kw, n, bias, dev):
    rng = np.random.default_rng(100 + n + E)
    l = (2 * rng.standard_normal((n, E))).astype(np.float32)
    compare(kw, l, (0.1 * rng.standard_normal(E)).astype(np.float32) if bias else None, dev)


@pytest.mark.parametrize("E,kw", ROUTES)
def test_route_masked(E, kw, dev):
    """Experts out by -inf, NaN and the lowest float, rows with fewer than k
    left, rows with none; a bias of -inf and NaN."""
    rng = np.random.default_rng(7)
    n = 120
    l = rng.standard_normal((n, E)).astype(np.float32)
    for p, value in ((0.2, -np.inf), (0.1, LOW), (0.05, np.nan)):
        l[rng.random((n, E)) < p] = value
    l[rng.random(n) < 0.1] = LOW
    l[rng.random(n) < 0.1] = -np.inf
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    compare(kw, l, None, dev)
    compare(kw, l, bias, dev)
    if E > 8:
        bias[3], bias[5] = -np.inf, np.nan
        compare(kw, l, bias, dev)


@pytest.mark.parametrize("E,kw", ROUTES)
def test_route_ties_take_the_lowest_index(E, kw, dev):
    rng = np.random.default_rng(8)
    l = rng.integers(-2, 3, size=(150, E)).astype(np.float32)
    compare(kw, l, None, dev)
    compare(kw, np.zeros((9, E), np.float32), None, dev)
    compare(kw, l, np.full(E, 0.25, np.float32), dev)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_chooses_as_in_64_bits(score, groups, dev):
    """Biased scores closer together than the rounding of FP32: logits one
    step of FP32 apart under one bias, and biases that undo the scores to
    within a rounding."""
    rng = np.random.default_rng(9)
    E, n = 32, 400
    base = rng.standard_normal((n, 1)).astype(np.float32)
    l = np.repeat(base, E, 1)
    for e in range(E):
        for _ in range(e % 5):
            l[:, e] = np.nextafter(l[:, e], np.float32(10))
    kw = dict(k=6, score=score, n_groups=groups, top_groups=min(groups, 2))
    compare(kw, l, np.full(E, 0.5, np.float32), dev)
    row = rng.standard_normal((1, E)).astype(np.float32)
    s = O.route_forward(row, None, 1, score)[4][0]
    bias = (1.0 - s).astype(np.float32)  # s + bias = 1 to a rounding, for the rows equal to `row`
    l = np.concatenate([np.repeat(row, 50, 0), (row + 1e-6 * rng.standard_normal((50, E))).astype(np.float32)])
    compare(kw, l, bias, dev)


def test_route_large_and_infinite_logits(dev):
    big = float(np.finfo(np.float32).max)
    l = np.array([[np.inf, 1.0, 2.0, np.inf], [big, big, 0.0, 1.0], [300.0, 200.0, -300.0, 0.0],
                  [-300.0, -301.0, -299.5, -400.0], [-3e38, -3.1e38, -np.inf, -3.2e38]], np.float32)
    for kw in (dict(k=2), dict(k=3, renormalise=False), dict(k=2, score="sigmoid", renormalise=False)):
        r = C().Router(4, **kw)
        ids, w, gates, _ = r.forward(T(l, dev))
        oi, ow, _, _, _ = O.route_forward(l, None, **kw)
        if kw.get("score") != "sigmoid":  # equal sigmoids: the order of the logits, which 64 bits no longer see
            assert np.array_equal(ids.cpu().numpy(), oi)
            assert np.all(np.abs(w.cpu().numpy() - ow) <= 160 * U * ow + 1e-37)
        assert torch.isfinite(w).all() and torch.isfinite(gates).all()
        d = r.backward(T(l, dev), ids, torch.ones_like(w))
        assert torch.isfinite(d).all()
    # chosen scores below the smallest float still share out the scale
    ids, w, _, _ = C().Router(4, 2, score="sigmoid").forward(T(l[3:4], dev))
    assert ids.tolist() == [[2, 0]]
    assert abs(w[0, 0].item() - 1 / (1 + np.exp(-0.5))) < 1e-6


def test_no_rows(dev):
    r = C().Router(6, 2)
    counts = torch.full((6,), 9, dtype=torch.int32, device=dev)
    ids, w, gates, c = r.forward(torch.empty(0, 6, device=dev), outs=(None, None, None, counts))
    assert not c.any()
    ids, w, gates, c = r.forward(torch.empty(0, 6, device=dev))
    assert ids.shape == (0, 2) and gates.shape == (6, 0) and not c.any()
    assert r.backward(torch.empty(0, 6, device=dev), ids, w).shape == (0, 6)


def test_partial_outputs_padding_and_guards(dev):
    rng = np.random.default_rng(10)
    n, E, k = 37, 12, 3
    r = C().Router(E, k, score="sigmoid", n_groups=4, top_groups=2)
    l = T(rng.standard_normal((n, E)).astype(np.float32), dev)
    full = r.forward(l)
    for want in (("ids",), ("weights",), ("gates",), ("counts",), ("ids", "gates")):
        for name, a, b in zip(("ids", "weights", "gates", "counts"), r.forward(l, want=want), full):
            assert (a is None) if name not in want else torch.equal(a, b), (want, name)
    assert all(full[2][e].data_ptr() % 16 == 0 and full[2][e].is_contiguous() for e in range(E))
    buf = torch.full((E, 48), 5.0, device=dev)
    r.forward(l, outs=(None, None, buf[:, :n], None))
    assert torch.equal(buf[:, :n], full[2]) and (buf[:, n:] == 5.0).all()  # columns behind the rows: as they were
    flat = torch.full((n * E + 128,), 5.0, device=dev)
    r.backward(l, full[0], full[1], buf[:, :n], grad_logits=flat[64:64 + n * E])
    assert (flat[:64] == 5.0).all() and (flat[64 + n * E:] == 5.0).all()
    ib, wb = torch.full((n * k + 64,), 7, dtype=torch.int32, device=dev), torch.full((n * k + 64,), 7.0, device=dev)
    r.forward(l, outs=(ib[32:32 + n * k], wb[32:32 + n * k], None, None))
    assert (ib[:32] == 7).all() and (ib[32 + n * k:] == 7).all() and (wb[32 + n * k:] == 7).all()
    assert torch.equal(ib[32:32 + n * k].view(n, k), full[0])
    with pytest.raises(C().CgtpError) as e:  # gates rows that are not 16-byte aligned
        r.forward(l, outs=(None, None, torch.empty(E, n, device=dev), None))
    assert e.value.status == 6


def test_backward_of_odd_ids(dev):
    """Ids outside the experts count as -1; a repeated id counts each time."""
    rng = np.random.default_rng(11)
    l = rng.standard_normal((4, 6)).astype(np.float32)
    ids = np.array([[0, 9, 2], [-5, -1, 1], [3, 3, 1], [2 ** 31 - 1, -2 ** 31, 5]], np.int32)
    gw = rng.standard_normal((4, 3)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            r = C().Router(6, 3, score=score, renormalise=renormalise)
            d = r.backward(T(l, dev), T(ids, dev), T(gw, dev)).cpu().numpy()
            ref = O.route_backward(l, ids, gw, None, score, renormalise)
            assert np.abs(d - ref).max() < 1e-6


def test_repeatable_graph_and_stream(dev):
    rng = np.random.default_rng(12)
    n, E = 5000, 64
    r = C().Router(E, 8, score="sigmoid", n_groups=8, top_groups=4)
    l, b = T(rng.standard_normal((n, E)).astype(np.float32), dev), T(0.1 * rng.standard_normal(E).astype(np.float32), dev)
    ref = r.forward(l, b)
    gg = T(rng.standard_normal((E, n)).astype(np.float32), dev)
    dref = r.backward(l, ref[0], grad_gates=gg)
    outs = [torch.full_like(t, 3) for t in ref[:2]] + [torch.full((E, n), 3.0, device=dev), torch.full_like(ref[3], 3)]
    d = torch.full_like(dref, 3)

    def step():
        r.forward(l, b, outs=outs)
        r.backward(l, outs[0], grad_gates=gg, grad_logits=d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    same = lambda: all(torch.equal(a, c) for a, c in zip(outs, ref)) and torch.equal(d, dref)
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for t in outs + [d]:
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert same()


def test_gradient_by_differences(dev):
    """<c, weights> along a random direction of the logits (choices kept)."""
    rng = np.random.default_rng(13)
    n, E, k = 200, 16, 4
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            r = C().Router(E, k, score=score, renormalise=renormalise)
            l = T((2 * rng.standard_normal((n, E))).astype(np.float32), dev)
            ids, w, _, _ = r.forward(l)
            c, v = (T(rng.standard_normal(s).astype(np.float32), dev) for s in ((n, k), (n, E)))
            h = 2e-3
            pi, pw, _, _ = r.forward(l + h * v)
            mi, mw, _, _ = r.forward(l - h * v)
            keep = ((pi == ids) & (mi == ids)).all(1)
            assert keep.float().mean().item() > 0.8
            num = ((pw - mw).double() * c.double()).sum(1) / (2 * h)
            d = (r.backward(l, ids, c).double() * v.double()).sum(1)
            # rounding 160 u |w| |c| / h <= 5e-3 a row at |w| <= 1, |c| ~ 2; truncation h^2 ~ 4e-6 of third derivatives
            assert (num - d)[keep].abs().max().item() < 2e-2
            assert ((num - d)[keep].norm() / d[keep].norm()).item() < 5e-3


def test_offsets_beyond_32_bits(dev):
    """2.2e9 logits and gates: the last rows equal the same rows alone."""
    n, E, k, m = 34_400_001, 64, 4, 3001
    gen = torch.Generator(device=dev)
    gen.manual_seed(2)
    tail, bias = torch.randn(m, E, device=dev, generator=gen), 0.1 * torch.randn(E, device=dev, generator=gen)
    l = torch.full((n, E), LOW, device=dev)
    l[-m:] = tail
    r = C().Router(E, k, score="sigmoid", n_groups=8, top_groups=3)
    ids, w, gates, counts = r.forward(l, bias)
    one = r.forward(tail, bias)
    assert torch.equal(ids[-m:], one[0]) and torch.equal(counts, one[3])
    # few rows are decided by warps, many by threads: the same choice, weights apart by both bounds
    assert ((w[-m:] - one[1]).abs() <= 320 * U * one[1]).all()
    assert torch.equal(gates[:, -m:] != 0, one[2] != 0) and not gates[:, :1000].any()
    assert (ids[:1000] == -1).all()
    d = r.backward(l, ids, grad_gates=gates)
    ref = r.backward(tail, one[0], grad_gates=one[2])
    assert ((d[-m:] - ref).abs() <= 1e-5).all() and not d[:1000].any()


def test_degenerate_rows_in_many(dev):
    """20,000 rows of equal logits, a router not yet trained: the lowest indices,
    on the form for many rows, with and without groups and bias."""
    for E, kw in ((64, dict(k=8, score="sigmoid", n_groups=8, top_groups=4)), (64, dict(k=8)), (24, dict(k=3, score="sigmoid"))):
        n = 20000
        l = torch.zeros(n, E, device=dev)
        for bias in (None, torch.zeros(E, device=dev)):
            ids, w, gates, counts = C().Router(E, **kw).forward(l, bias)
            oi, ow, _, _, _ = O.route_forward(np.zeros((1, E), np.float32), None if bias is None else np.zeros(E), **kw)
            assert (ids.cpu().numpy() == oi).all()
            assert np.abs(w.cpu().numpy() - ow).max() <= 160 * U
            assert counts.sum().item() == n * kw["k"]


@pytest.mark.parametrize("E,kw", ROUTES)
def test_route_many_rows(E, kw, dev):
    """The form for many rows against the oracle, whose rows are drawn from a
    short list (the oracle goes row by row)."""
    rng = np.random.default_rng(14)
    base = (2 * rng.standard_normal((150, E))).astype(np.float32)
    base[rng.random((150, E)) < 0.1] = -np.inf
    base[7] = LOW
    pick = rng.integers(0, 150, size=20001)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, bias):
        oi, ow, _, _, _ = O.route_forward(base, b, **kw)
        ids, w, gates, counts = C().Router(E, **kw).forward(T(base[pick], dev), None if b is None else T(b, dev))
        assert np.array_equal(ids.cpu().numpy(), oi[pick])
        assert np.all(np.abs(w.cpu().numpy() - ow[pick]) <= 160 * U * ow[pick] + 1e-38)
        assert np.array_equal(counts.cpu().numpy(), np.bincount(oi[pick][oi[pick] >= 0], minlength=E))
        ref = np.zeros((E + 1, len(pick)), np.float32)
        ref[np.where(oi[pick] < 0, E, oi[pick]), np.arange(len(pick))[:, None]] = w.cpu().numpy()
        assert np.array_equal(gates.cpu().numpy(), ref[:E])


@pytest.mark.parametrize("n", [150, 20001])
@pytest.mark.parametrize("E,kw", [(75, dict(k=8, score="sigmoid", renormalise=False)), (75, dict(k=5)), (24, dict(k=1)),
                                  (64, dict(k=8, score="sigmoid", n_groups=8, top_groups=4)),
                                  (64, dict(k=3, score="softmax", n_groups=4, top_groups=2, group_best=1))])
def test_route_of_close_logits(E, kw, n, dev):
    """A dozen logits of every row a few steps of FP32 apart, in any order: the
    FP32 forms meet wrong orders and decide them in 64 bits."""
    rng = np.random.default_rng(15)
    base = rng.standard_normal((150, E)).astype(np.float32)
    for t in range(150):
        at = rng.choice(E, 12, replace=False)
        base[t, at] = 3 + rng.integers(0, (4, 40, 400)[t % 3], 12) * np.float32(2.0 ** -22)
    pick = np.arange(n) % 150
    for b in (None, np.full(E, 0.125, np.float32), (1e-7 * rng.standard_normal(E)).astype(np.float32)):
        oi, ow, _, _, _ = O.route_forward(base, b, **kw)
        ids, w, _, _ = C().Router(E, **kw).forward(T(base[pick], dev), None if b is None else T(b, dev))
        assert np.array_equal(ids.cpu().numpy(), oi[pick])
        assert np.all(np.abs(w.cpu().numpy() - ow[pick]) <= 160 * U * ow[pick] + 1e-38)


def test_gradient_of_a_single_choice_is_zero(dev):
    """Renormalised, one expert's weight is the scale whatever its logit."""
    rng = np.random.default_rng(16)
    for score in ("softmax", "sigmoid"):
        for E, n in ((5, 300), (64, 70000)):
            l = T(rng.standard_normal((n, E)).astype(np.float32), dev)
            r = C().Router(E, 1, score=score, scale=2.5)
            ids, w, _, _ = r.forward(l)
            assert (w == 2.5).all()
            assert not r.backward(l, ids, torch.randn_like(w)).any()


def test_backward_ignores_the_gradient_of_what_is_out(dev):
    """A NaN in the gradient at an id that is -1, or whose logit is masked, reaches nothing."""
    rng = np.random.default_rng(17)
    l = rng.standard_normal((6, 8)).astype(np.float32)
    l[1, 2], l[2, 2], l[3, 2] = -np.inf, np.nan, LOW
    ids = np.tile(np.array([[1, 2, 5]], np.int32), (6, 1))
    ids[4, 1] = -1
    gw = rng.standard_normal((6, 3)).astype(np.float32)
    gw[1:5, 1] = np.nan
    clean = np.where(np.isnan(gw), 0, gw).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            r = C().Router(8, 3, score=score, renormalise=renormalise)
            d = r.backward(T(l, dev), T(ids, dev), T(gw, dev)).cpu().numpy()
            ref = O.route_backward(l, ids, clean, None, score, renormalise)
            assert np.abs(d - ref).max() < 1e-6


@pytest.mark.parametrize("E,kw", [(64, dict(k=8)), (64, dict(k=8, renormalise=False)), (16, dict(k=4)), (40, dict(k=5, n_groups=4, top_groups=2)),
                                  (40, dict(k=5, n_groups=4, top_groups=2, renormalise=False)), (24, dict(k=8, score="sigmoid")),
                                  (64, dict(k=8, score="sigmoid", n_groups=8, top_groups=4)), (128, dict(k=8, scale=3.0))])
def test_weights_of_small_scores(E, kw, dev):
    """Logits far apart, and a bias that steers to the small scores (some below
    the smallest float): each weight within the bound of its own size, on the
    form for few rows and on the one for many."""
    rng = np.random.default_rng(21)
    base = (rng.choice([1.0, 20.0, 45.0], size=(200, 1)) * rng.standard_normal((200, E))).astype(np.float32)
    base[::3] -= 40
    bias = np.where(rng.random(E) < 0.5, 2.0, -2.0).astype(np.float32) + (0.1 * rng.standard_normal(E)).astype(np.float32)
    oi, ow, _, _, _ = O.route_forward(base, bias, **kw)
    for pick in (np.arange(200), rng.integers(0, 200, size=20001)):
        ids, w, _, _ = C().Router(E, **kw).forward(T(base[pick], dev), T(bias, dev))
        assert np.array_equal(ids.cpu().numpy(), oi[pick])
        assert np.all(np.abs(w.cpu().numpy() - ow[pick]) <= 160 * U * ow[pick] + kw.get("scale", 1.0) * 1.2e-38)


@pytest.mark.parametrize("E,kw", [(4, dict(k=1, renormalise=False)), (16, dict(k=2)), (32, dict(k=4, score="sigmoid")),
                                  (12, dict(k=4, n_groups=12, top_groups=5))])
@pytest.mark.parametrize("bias", [False, True])
def test_route_more_rows_than_a_wave(E, kw, bias, dev):
    """Short rows, so many that a CTA takes several tiles: as the same rows in
    parts that it takes at once."""
    n, part = 300_001, 60_000
    gen = torch.Generator(device=dev)
    gen.manual_seed(5)
    l = torch.randn(n, E, device=dev, generator=gen)
    l[torch.rand(n, E, device=dev, generator=gen) < 0.1] = LOW
    b = 0.1 * torch.randn(E, device=dev, generator=gen) if bias else None
    r = C().Router(E, **kw)
    ids, w, gates, counts = r.forward(l, b)
    total = torch.zeros(E, dtype=torch.int32, device=dev)
    for t in range(0, n, part):
        i, v, g, c = r.forward(l[t:t + part].clone(), b)
        assert torch.equal(ids[t:t + part], i)
        # the last part, one row, is decided by the form for few rows: each form's weights are
        # within 160 u of the exact ones, so within 320 u of the other's; else the same bits
        u = 320 * U if len(i) < part else 0.0
        assert ((w[t:t + part] - v).abs() <= u * v).all() and ((gates[:, t:t + part] - g).abs() <= u * g).all()
        total += c
    assert torch.equal(counts, total)
