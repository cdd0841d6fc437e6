"""GPU parity of the router where its forms could part from the definition:
zeros of both signs, biases of the lowest float, saturated sigmoids, and
gradients of a row whose weight lies almost all on one expert.

Choices are equal to the FP64 oracle's.  A weight is off by at most 160 u of
itself (the parity tests count its roundings).  The gradients' bound: with
the shares p of a row and any constant c, sum p d is c + sum p (d - c), so a
logit's gradient is
  w (d - c - sum p (d - c))
whatever c; with c the d of an expert that holds more than half of the row it
has no terms that cancel as a whole.  Shares are off by 160 u of themselves, the
differences and the sum of at most 64 terms by less than that again: 320 u of
w (|d - c| + sum p |d - c|), and (1 - p) of a sigmoid, formed from its logit,
is inside that too.
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


def choices(l, bias, kw, dev, n):
    """The kernel's ids, weights, gates and counts of n rows drawn in turn from
    l's against the oracle's."""
    pick = np.arange(n) % len(l)
    oi, ow, _, _, _ = O.route_forward(l, bias, **kw)
    E = l.shape[1]
    ids, w, gates, counts = C().Router(E, **kw).forward(T(l[pick], dev), None if bias is None else T(bias, dev))
    assert np.array_equal(ids.cpu().numpy(), oi[pick])
    assert np.all(np.abs(w.cpu().numpy() - ow[pick]) <= 160 * U * ow[pick] + kw.get("scale", 1.0) * 1.2e-38)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(oi[pick][oi[pick] >= 0], minlength=E))
    ref = np.zeros((E + 1, n), np.float32)
    ref[np.where(oi[pick] < 0, E, oi[pick]), np.arange(n)[:, None]] = w.cpu().numpy()
    assert np.array_equal(gates.cpu().numpy(), ref[:E])


@pytest.mark.parametrize("n", [60, 20001])
@pytest.mark.parametrize("E,kw", [(4, dict(k=1)), (4, dict(k=2, renormalise=False)), (24, dict(k=3, score="sigmoid")),
                                  (64, dict(k=8)), (64, dict(k=12)), (75, dict(k=5, score="sigmoid", renormalise=False)),
                                  (200, dict(k=4, renormalise=False))])
def test_zeros_of_both_signs_are_equal(E, kw, n, dev):
    """Logits times a mask of zeros and ones: -0.0 and 0.0 are one value, and the
    lowest index goes first, also across the cut of the k best."""
    rng = np.random.default_rng(31)
    l = rng.standard_normal((60, E)).astype(np.float32)
    l *= rng.random((60, E)) < np.linspace(0, 0.6, 60)[:, None]  # a negative logit's zero is -0.0
    l[0, :4] = [-0.0, 0.0, -1.0, 0.0]
    l[0, 4:] = -1.0
    l[1] = np.where(np.arange(E) % 2 == 0, -0.0, 0.0)
    assert np.signbit(l[l == 0]).any() and not np.signbit(l[l == 0]).all()
    choices(l, None, kw, dev, n)
    choices(l, np.where(np.arange(E) % 3 == 0, -0.0, 0.0).astype(np.float32), kw, dev, n)


@pytest.mark.parametrize("n", [60, 20001])
@pytest.mark.parametrize("kw", [dict(k=8, score="sigmoid"), dict(k=8, renormalise=False), dict(k=12)])
def test_biases_of_the_lowest_float(kw, n, dev):
    """A bias of the lowest float puts an expert last, it does not rule it out: a
    group of two such experts, whose sum is below the lowest float, can be chosen."""
    rng = np.random.default_rng(32)
    kw = dict(kw, n_groups=8, top_groups=4)
    l = rng.standard_normal((60, 32)).astype(np.float32)
    for open_experts in ([0, 2], [13, 14, 30], [], list(range(24))):
        bias = np.full(32, LOW, np.float32)
        bias[open_experts] = 0.1 * rng.standard_normal(len(open_experts))
        choices(l, bias, kw, dev, n)
        bias[1::4] = -np.inf  # one of every group out
        choices(l, bias, kw, dev, n)


def shifted(l, ids, d, kw):
    """The gradient's magnitudes [rows, E] by the module's bound, for d [rows, k]."""
    n, E = l.shape
    scale, renormalise, sigmoid = kw.get("scale", 1.0), kw.get("renormalise", True), kw.get("score") == "sigmoid"
    z = l.astype(np.float64)
    p = np.exp(z - z.max(1, keepdims=True))
    p = 1 / (1 + np.exp(-z)) if sigmoid else p / p.sum(1, keepdims=True)
    de, chosen = np.zeros((n, E)), np.zeros((n, E), bool)
    np.put_along_axis(de, ids, d.astype(np.float64), 1)
    np.put_along_axis(chosen, ids, True, 1)
    share = np.where(chosen, p, 0) if renormalise else p
    share = share / share.sum(1, keepdims=True)
    top = share.argmax(1)[:, None]
    c = np.where(np.take_along_axis(share, top, 1) > 0.5, np.take_along_axis(de, top, 1), 0.0)
    mag = scale * share * (np.abs(de - c) + (share * np.abs(de - c)).sum(1, keepdims=True))
    return mag * (1 - p) if sigmoid else mag


def dominant(n, E, seed):
    """Rows with one logit some 3 to 15 above the others."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((n, E)).astype(np.float32)
    l[np.arange(n), rng.integers(0, E, n)] += np.linspace(3, 15, n, dtype=np.float32)
    return rng, l


@pytest.mark.parametrize("E,kw", [(64, dict(k=12)), (40, dict(k=32, scale=2.5)), (200, dict(k=9)), (64, dict(k=8)), (5, dict(k=2)),
                                  (64, dict(k=12, score="sigmoid"))])
def test_gradient_of_a_dominant_share(E, kw, dev):
    """Renormalised: next to a share of 1 - 1e-6 each gradient is right to its own
    size, not to that of the d it is formed from."""
    rng, l = dominant(200, E, 33)
    if kw.get("score") == "sigmoid":  # shares of e^(l - largest) / (1 + e^l)
        l -= 12
    r = C().Router(E, **kw)
    ids = r.forward(T(l, dev))[0].cpu().numpy()
    d = (1 + 0.1 * rng.standard_normal(ids.shape)).astype(np.float32)
    got = r.backward(T(l, dev), T(ids, dev), T(d, dev)).cpu().numpy().astype(np.float64)
    ref = O.route_backward(l, ids, d, None, **{k: v for k, v in kw.items() if k in ("score", "renormalise", "scale")})
    mag = shifted(l, ids, d, kw)
    assert (np.abs(got - ref) <= 320 * U * mag + 1e-37).all(), float((np.abs(got - ref) / (U * mag + 1e-37)).max())


@pytest.mark.parametrize("E,k", [(3, 2), (8, 1), (16, 2), (30, 5), (64, 8), (100, 3), (200, 32), (512, 4)])
def test_gradient_of_a_dominant_score(E, k, dev):
    """The plain softmax, where the dominant expert is among the chosen (the first
    of them) and where it is not."""
    rng, l = dominant(200, E, 34)
    kw = dict(k=k, renormalise=False, scale=1.5)
    r = C().Router(E, **kw)
    first = r.forward(T(l, dev))[0].cpu().numpy()
    other = np.argsort(l, 1)[:, :k].astype(np.int32)
    for ids in (first, other):
        d = (1 + 0.1 * rng.standard_normal(ids.shape)).astype(np.float32)
        got = r.backward(T(l, dev), T(ids, dev), T(d, dev)).cpu().numpy().astype(np.float64)
        ref = O.route_backward(l, ids, d, None, renormalise=False, scale=1.5)
        mag = shifted(l, ids, d, kw)
        assert (np.abs(got - ref) <= 320 * U * mag + 1e-37).all(), float((np.abs(got - ref) / (U * mag + 1e-37)).max())


def test_dominant_score_listed_twice(dev):
    """Each place of a repeated id counts, also of the dominant one's."""
    rng, l = dominant(200, 16, 35)
    top = l.argmax(1)
    ids = np.stack([top, top, (top + 1) % 16, top], 1).astype(np.int32)
    d = rng.standard_normal(ids.shape).astype(np.float32)
    r = C().Router(16, 4, renormalise=False)
    got = r.backward(T(l, dev), T(ids, dev), T(d, dev)).cpu().numpy().astype(np.float64)
    ref = O.route_backward(l, ids, d, None, renormalise=False)
    # as one place with the sum of the three, itself off by 2 u of the sum of magnitudes
    mag = shifted(l, ids[:, 1:3], np.stack([d[:, [0, 1, 3]].sum(1), d[:, 2]], 1), dict(renormalise=False))
    p = np.exp(l - l.max(1, keepdims=True).astype(np.float64))
    p /= p.sum(1, keepdims=True)
    mag += 2 / 320 * np.abs(d).sum(1, keepdims=True) * p * np.where(np.arange(16) == top[:, None], 1 - p, 1)
    assert (np.abs(got - ref) <= 320 * U * mag + 1e-37).all(), float((np.abs(got - ref) / (U * mag + 1e-37)).max())


def test_large_logits_of_sigmoids(dev):
    """Saturated sigmoids are chosen by their logits, infinite ones as the
    largest float; those below the smallest float keep their order."""
    big = float(np.finfo(np.float32).max)
    l = np.array([[np.inf, 1.0, 2.0, np.inf], [big, big, 0.0, 1.0], [300.0, 200.0, -300.0, 0.0],
                  [-300.0, -301.0, -299.5, -400.0], [-3e38, -3.1e38, -np.inf, -3.2e38]], np.float32)
    for k in (1, 2, 3):
        for n in (5, 20000):
            choices(l, None, dict(k=k, score="sigmoid", renormalise=False), dev, n)
            choices(l[:4], None, dict(k=k, score="sigmoid"), dev, n)
