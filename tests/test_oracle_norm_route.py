"""Pins of the oracle's layer norm of irreps rows and of its router (CPU).

The norm against torch's layer norm and against its own definition on one
block, its equivariance under rotations and inversion, its first and second
derivatives against central differences, with a planted mistake that fails.
The router against a brute-force choice, ties, masked experts and rows,
groups, and its gradient against central differences of <weights, c> with the
choice held fixed.
"""
import itertools

import numpy as np
import pytest

import oracle as O
from tests._so3 import block_rotation, random_rotation

EPS = 1e-5
IRREPS = ["9x0e", "7x0e+5x1o+3x2e+1x3o", "3x0o+4x0e+2x0e+2x6e", "1x0e+1x0o+1x1e"]


def dims(irreps):
    b = O.parse_irreps(irreps)
    return O.dim(b), sum(m for m, _, _ in b), sum(m for m, l, p in b if l == 0 and p > 0)


def draw(irreps, n, seed):
    rng = np.random.default_rng(seed)
    D, C, S = dims(irreps)
    return (rng.standard_normal((n, D)) + 0.4, 1 + 0.3 * rng.standard_normal(C), rng.standard_normal(S),
            rng.standard_normal((n, D)))


def test_norm_of_scalars_is_the_plain_layer_norm():
    torch = pytest.importorskip("torch")
    x, w, b, _ = draw("37x0e", 5, 0)
    t = lambda a: torch.from_numpy(a)
    ref = torch.nn.functional.layer_norm(t(x), (37,), t(w), t(b), EPS).numpy()
    assert np.abs(O.norm_forward("37x0e", x, w, b, EPS) - ref).max() < 1e-13


def test_norm_of_vectors_has_unit_mean_square():
    x, _, _, _ = draw("6x2o", 4, 1)
    y = O.norm_forward("6x2o", x, np.ones(6), np.zeros(0), 1e-12)
    assert np.abs((y ** 2).mean(1) - 1).max() < 1e-11
    assert np.abs(y / x - (y / x)[:, :1]).max() < 1e-12  # one factor a row: directions kept


@pytest.mark.parametrize("irreps", IRREPS)
@pytest.mark.parametrize("parity", [1, -1])
def test_norm_equivariance(irreps, parity):
    x, w, b, _ = draw(irreps, 3, 2)
    R = random_rotation(np.random.default_rng(3))
    M = block_rotation(O.parse_irreps(irreps), R, parity)
    a = O.norm_forward(irreps, x @ M.T, w, b, EPS)
    assert np.abs(a - O.norm_forward(irreps, x, w, b, EPS) @ M.T).max() < 1e-10


def test_centring_a_vector_block_would_break_equivariance():
    """The pin above catches it: a norm that also centres l > 0 blocks."""
    x, w, _, _ = draw("5x1o", 3, 4)
    M = block_rotation(O.parse_irreps("5x1o"), random_rotation(np.random.default_rng(5)))
    f = lambda z: O.norm_forward("15x0e", z, np.repeat(w, 3), np.zeros(15), EPS)
    assert np.abs(f(x @ M.T) - f(x) @ M.T).max() > 1e-2


def central(f, z, h=1e-6):
    g = np.zeros_like(z)
    for i in itertools.product(*(range(s) for s in z.shape)):
        p, m = z.copy(), z.copy()
        p[i] += h
        m[i] -= h
        g[i] = (f(p) - f(m)) / (2 * h)
    return g


@pytest.mark.parametrize("irreps", IRREPS)
def test_norm_backward_is_the_difference_quotient(irreps):
    x, w, b, g = draw(irreps, 3, 6)
    L = lambda x_, w_, b_: float((O.norm_forward(irreps, x_, w_, b_, EPS) * g).sum())
    dx, dw, db = O.norm_backward(irreps, x, w, g, EPS)
    # blocks of one value (1x0e, 1x0o) have gradients of the order of eps
    assert np.abs(dx - central(lambda z: L(z, w, b), x)).max() < 1e-7
    assert np.abs(dw - central(lambda z: L(x, z, b), w)).max() < 1e-7
    assert np.abs(db - central(lambda z: L(x, w, z), b)).max() < 1e-7 if len(b) else db.size == 0


@pytest.mark.parametrize("irreps", IRREPS)
def test_norm_double_backward_is_the_difference_quotient(irreps):
    x, w, b, g = draw(irreps, 2, 7)
    hx, hw, hb, _ = draw(irreps, 2, 8)

    def S(g_, x_, w_):
        dx, dw, db = O.norm_backward(irreps, x_, w_, g_, EPS)
        return float((hx * dx).sum() + (hw * dw).sum() + (hb * db).sum())
    gg, gx, gw = O.norm_double_backward(irreps, x, w, g, hx, hw, hb, EPS)
    for got, ref in ((gg, central(lambda z: S(z, x, w), g)), (gx, central(lambda z: S(g, z, w), x)),
                     (gw, central(lambda z: S(g, x, z), w))):
        assert np.abs(got - ref).max() < 2e-6 * max(1.0, np.abs(ref).max())


def test_pins_catch_a_dropped_term():
    x, w, b, g = draw("9x0e", 3, 9)
    xh, r = O.norm_forward("9x0e", x, np.ones(9), np.zeros(9), EPS), None
    L = lambda z: float((O.norm_forward("9x0e", z, w, b, EPS) * g).sum())
    a = g * w
    r = 1 / np.sqrt(x.var(1, keepdims=True) + EPS)
    wrong = r * (a - xh * (a * xh).mean(1, keepdims=True))  # without mean(a)
    assert np.abs(wrong - central(L, x)).max() > 1e-2


# ---- router
ROUTES = [dict(k=1, score="softmax", renormalise=False), dict(k=3, score="softmax", renormalise=True, scale=2.5),
          dict(k=2, score="sigmoid", renormalise=False), dict(k=4, score="sigmoid", renormalise=True),
          dict(k=3, score="sigmoid", n_groups=4, top_groups=2, group_best=2),
          dict(k=2, score="softmax", n_groups=3, top_groups=1, group_best=1, renormalise=False)]


@pytest.mark.parametrize("kw", ROUTES)
def test_route_choice_is_the_best_subset(kw):
    """Without groups the chosen set has the largest sum of biased scores of
    all sets of k; with groups, of all sets inside top_groups groups."""
    rng = np.random.default_rng(10)
    E, n = 12, 6
    l, bias = rng.standard_normal((n, E)), 0.2 * rng.standard_normal(E)
    ids, w, gates, counts, s = O.route_forward(l, bias, **kw)
    e = np.exp(l)
    ref = e / e.sum(1, keepdims=True) if kw["score"] == "softmax" else e / (1 + e)
    assert np.abs(s - ref).max() < 1e-14
    G, T, m = kw.get("n_groups", 1), kw.get("top_groups", 1), kw.get("group_best", 2)
    for t in range(n):
        v = ref[t] + bias
        part = v.reshape(G, -1)
        sets = itertools.combinations(range(G), T)
        best = max(sets, key=lambda q: sum(np.sort(part[g])[::-1][:m].sum() for g in q)) if G > 1 else (0,)
        pool = [i for i in range(E) if i // (E // G) in best]
        top = max(itertools.combinations(pool, kw["k"]), key=lambda q: v[list(q)].sum())
        assert set(ids[t]) == set(top)
        assert np.all(np.diff(v[ids[t]]) <= 0)
        p = ref[t][ids[t]]
        want = kw.get("scale", 1.0) * (p / p.sum() if kw.get("renormalise", True) else p)
        assert np.abs(w[t] - want).max() < 1e-14
        assert np.array_equal(np.flatnonzero(gates[:, t]), np.sort(ids[t]))
    assert np.array_equal(counts, np.bincount(ids.ravel(), minlength=E))


def test_route_masks_ties_and_empty_rows():
    low = float(np.finfo(np.float32).min)
    l = np.array([[1.0, 1.0, 1.0, 1.0], [-np.inf, 0.5, low, np.nan], [-np.inf, low, np.nan, -np.inf],
                  [np.inf, 2.0, np.inf, 0.0]])
    ids, w, gates, counts, s = O.route_forward(l, None, 2)
    assert ids.tolist() == [[0, 1], [1, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]
    assert counts.tolist() == [2, 2, 1, 0]
    assert not gates[:, 2].any() and not s[2].any()
    ids, _, _, _, _ = O.route_forward(l[:1], [-np.inf, 0.0, np.nan, 0.0], 3)  # a bias that rules experts out
    assert ids.tolist() == [[1, 3, -1]]


@pytest.mark.parametrize("kw", ROUTES)
def test_route_backward_is_the_difference_quotient(kw):
    rng = np.random.default_rng(11)
    E, n = 12, 4
    l = rng.standard_normal((n, E))
    l[1, 3] = -np.inf
    l[2, :] = float(np.finfo(np.float32).min)
    ids, w, _, _, _ = O.route_forward(l, None, **kw)
    c, cg = rng.standard_normal(w.shape), rng.standard_normal((E, n))
    back = {k: v for k, v in kw.items() if k in ("score", "renormalise", "scale")}
    d = O.route_backward(l, ids, c, cg, **back)

    def L(z):
        e = np.where(z > np.finfo(np.float32).min, np.exp(np.where(z > -1e30, z, 0)), 0.0)
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300) if kw["score"] == "softmax" else e / (1 + e)
        p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
        if kw.get("renormalise", True):
            p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
        dd = c + np.where(ids >= 0, cg[np.maximum(ids, 0), np.arange(n)[:, None]], 0.0)
        return kw.get("scale", 1.0) * float((p * dd).sum())
    live = l > -1e30
    num = np.zeros_like(l)
    for i in zip(*np.nonzero(live)):
        p, m = l.copy(), l.copy()
        p[i] += 1e-6
        m[i] -= 1e-6
        num[i] = (L(p) - L(m)) / 2e-6
    assert np.abs(d - num).max() < 1e-8
    assert not d[~live].any()
