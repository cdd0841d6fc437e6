"""GPU parity of the layer norm of irreps rows against the FP64 oracle.

Tolerances.  u = 2^-24.  A block's sums run over its N values in partial sums
of at most 64 terms a thread, then a tree: each sum is off by at most (64 + 16)
u of the sum of magnitudes.  Element by element, an output is a short formula
in such sums; its error is at most K u times the sum of the magnitudes of the
formula's terms, each divided by its mean's cancellation: with m = (|x| +
mean|x|) r standing for |xh| (its subtraction cancels), K = 160 covers two
chained sums.  The weights' gradients add rows in chains of at most 700 terms
here, (700 + 80) u of the sum of magnitudes.
"""
import numpy as np
import pytest

import oracle as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5
U = 2.0 ** -24
K = 160


def C():
    from equivariant_mlip_clebsch_b200 import cgtp
    return cgtp


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def T(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def dims(irreps):
    b = O.parse_irreps(irreps)
    return O.dim(b), sum(m for m, _, _ in b), sum(m for m, l, p in b if l == 0 and p > 0)


def draw(irreps, n, seed, offset=0.3):
    rng = np.random.default_rng(seed)
    D, Cn, S = dims(irreps)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    x = (f(n, D) * np.exp(0.5 * f(n, 1)) + offset).astype(np.float32)
    return dict(x=x, w=1 + 0.3 * f(Cn), b=f(S), g=f(n, D), hx=f(n, D), hw=0.3 * f(Cn), hb=f(S))


def magnitudes(irreps, v, n):
    """Elementwise sums of term magnitudes: of y, grad_x, gg, gx and, per
    channel, of grad_weight, grad_bias, gweight."""
    a64 = lambda k: np.abs(v[k].astype(np.float64))
    x, g, h = v["x"].astype(np.float64), a64("g"), a64("hx")
    out = {k: np.zeros_like(x) for k in ("y", "dx", "gg", "gx")}
    out["dw"], out["gw"], out["db"] = np.zeros(len(v["w"])), np.zeros(len(v["w"])), []
    for cs, ws, bs, d in O.oracle._norm_blocks(irreps):
        _, r = O.oracle._norm_stats(x, cs, bs is not None, EPS)
        M = lambda z: z.mean(1, keepdims=True)
        W, HW = np.repeat(a64("w")[ws], d), np.repeat(a64("hw")[ws], d)
        ax = np.abs(x[:, cs])
        xh = (ax + (M(ax) if bs is not None else 0)) * r
        A, H, Kk = W * g[:, cs], h[:, cs], HW * g[:, cs]
        P = lambda z: z + (M(z) if bs is not None else 0)
        J = lambda z: r * (P(z) + xh * M(P(z) * xh))
        out["y"][:, cs] = xh * W + (a64("b")[bs] if bs is not None else 0)
        out["dx"][:, cs] = J(A)
        out["gg"][:, cs] = W * J(H) + HW * xh + (a64("hb")[bs] if bs is not None else 0)
        al, be = M(P(A) * xh), M(P(H) * xh)
        out["gx"][:, cs] = r * r * (xh * (3 * al * be + M(P(H) * A)) + be * P(A) + al * P(H)) + J(Kk)
        out["dw"][ws] = (g[:, cs] * xh).sum(0).reshape(-1, d).sum(1)
        out["gw"][ws] = (g[:, cs] * J(H)).sum(0).reshape(-1, d).sum(1)
        if bs is not None:
            out["db"].append(g[:, cs].sum(0))
    out["db"] = np.concatenate(out["db"]) if out["db"] else np.zeros(0)
    return out


def close(got, ref, mag, k, what):
    got = got.cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, what
    bad = np.abs(got - ref) - k * U * mag
    assert not np.isnan(got).any() and (bad.size == 0 or bad.max() <= 0), (what, float(np.nanmax(bad)))


def check(irreps, n, seed, dev, offset=0.3):
    v = draw(irreps, n, seed, offset)
    d = {k: T(a, dev) for k, a in v.items()}
    norm = C().LayerNorm(irreps, EPS)
    mag = magnitudes(irreps, v, n)
    y = norm.forward(d["x"], d["w"], d["b"])
    close(y, O.norm_forward(irreps, v["x"], v["w"], v["b"], EPS), mag["y"], K, "y")
    dx, dw, db = norm.backward(d["x"], d["w"], d["g"])
    rx, rw, rb = O.norm_backward(irreps, v["x"], v["w"], v["g"], EPS)
    close(dx, rx, mag["dx"], K, "grad_x")
    close(dw, rw, mag["dw"], K + 700, "grad_weight")
    close(db, rb, mag["db"], K + 700, "grad_bias")
    gg, gx, gw = norm.double_backward(d["x"], d["w"], d["g"], d["hx"], d["hw"], d["hb"])
    rg, rx, rw = O.norm_double_backward(irreps, v["x"], v["w"], v["g"], v["hx"], v["hw"], v["hb"], EPS)
    close(gg, rg, mag["gg"], K, "grad_grad")
    close(gx, rx, mag["gx"], 2 * K, "second grad_x")  # products of two sums
    close(gw, rw, mag["gw"], K + 700, "second grad_weight")
    return norm, v, d


IRREPS = ["1x0e", "64x0e", "7x0e+5x1o+3x2e+1x3o", "37x0e+21x1o+11x2e", "128x0e+64x1o+32x2e+32x3o",
          "3x0o+4x0e+2x0e+9x6e", "4x0e+1x1o", "1100x0e+340x3o", "2048x0e+12x1e", "33x0e+511x1o", "8x0e+4x1o+4x0e+8x2e"]


@pytest.mark.parametrize("irreps", IRREPS)
@pytest.mark.parametrize("n", [1, 2, 33, 700])
def test_norm_matches_the_oracle(irreps, n, dev):
    check(irreps, n, 20 + n, dev)


@pytest.mark.parametrize("irreps,n", [("1024x6e", 9), ("5001x1o", 5), ("20000x0e", 7), ("16385x0e+4x0e", 3),
                                      ("7001x2o", 4), ("40000x0e+10000x1o", 2), ("4096x0e", 40), ("4097x0e", 40),
                                      ("448x0e+768x1o+1024x2e+1152x3o+1216x4e+1152x5o+1024x6e", 5)])
def test_norm_of_wide_blocks(irreps, n, dev):
    check(irreps, n, 3, dev)


def test_norm_far_offset(dev):
    """Values 1000 from zero: centred in two passes, not by mean squares."""
    check("64x0e+512x0e", 50, 5, dev, offset=1000.0)


def test_many_rows_sum_to_the_weights_gradient(dev):
    """20,000 short rows: chains of rows per thread stay short (a sum over
    rows is split at least 100 ways), so the bound of 780 u holds."""
    n = 20000
    v = draw("12x0e+5x1o", n, 6)
    d = {k: T(a, dev) for k, a in v.items()}
    norm = C().LayerNorm("12x0e+5x1o", EPS)
    _, dw, db = norm.backward(d["x"], d["w"], d["g"], want=("weight", "bias"))
    _, rw, rb = O.norm_backward("12x0e+5x1o", v["x"], v["w"], v["g"], EPS)
    mag = magnitudes("12x0e+5x1o", v, n)
    close(dw, rw, mag["dw"], K + 700, "grad_weight")
    close(db, rb, mag["db"], K + 700, "grad_bias")


def test_no_rows(dev):
    norm = C().LayerNorm("8x0e+4x1o")
    x, w, b = torch.empty(0, 20, device=dev), torch.ones(12, device=dev), torch.ones(8, device=dev)
    assert norm.forward(x, w, b).shape == (0, 20)
    dw, db, gw = (torch.full((m,), 7.0, device=dev) for m in (12, 8, 12))
    norm.backward(x, w, x, grads=(torch.empty(0, 20, device=dev), dw, db))
    norm.double_backward(x, w, x, h_x=x, grads=(None, None, gw))
    assert not dw.any() and not db.any() and not gw.any()


def test_defaults_and_partial_outputs(dev):
    irreps = "20x0e+6x1o+3x0o"
    norm, v, d = check(irreps, 21, 7, dev)
    one, zero = np.ones_like(v["w"]), np.zeros_like(v["b"])
    mag = magnitudes(irreps, dict(v, w=one, b=zero), 21)
    close(norm.forward(d["x"]), O.norm_forward(irreps, v["x"], one, zero, EPS), mag["y"], K, "y")
    full = norm.backward(d["x"], d["w"], d["g"])
    for want in (("x",), ("weight",), ("bias",), ("x", "bias")):
        got = norm.backward(d["x"], d["w"], d["g"], want=want)
        for name, a, b in zip(("x", "weight", "bias"), got, full):
            assert (a is None) if name not in want else torch.equal(a, b), (want, name)
    rx, _, _ = O.norm_backward(irreps, v["x"], one, v["g"], EPS)
    close(norm.backward(d["x"], None, d["g"])[0], rx, mag["dx"], K, "grad_x without weight")
    args = dict(hx=d["hx"], hw=d["hw"], hb=d["hb"])
    for keys in ((), ("hx",), ("hw",), ("hb",), ("hx", "hw"), ("hw", "hb")):
        h = {k: (a if k in keys else None) for k, a in args.items()}
        ref = O.norm_double_backward(irreps, v["x"], v["w"], v["g"], *(v[k] if k in keys else np.zeros_like(v[k])
                                                                       for k in ("hx", "hw", "hb")), EPS)
        got = norm.double_backward(d["x"], d["w"], d["g"], h["hx"], h["hw"], h["hb"])
        m = magnitudes(irreps, v, 21)
        for a, r, mm, k in zip(got, ref, (m["gg"], m["gx"], m["gw"]), (K, 2 * K, K + 700)):
            close(a, r, mm, k, keys)
        for want in (("g",), ("x",), ("weight",)):
            part = norm.double_backward(d["x"], d["w"], d["g"], h["hx"], h["hw"], h["hb"], want=want)
            for name, a, b in zip(("g", "x", "weight"), part, got):
                assert (a is None) if name not in want else torch.equal(a, b), (keys, want)


def test_non_finite_values_stay_in_their_block(dev):
    irreps = "16x0e+8x1o"
    v = draw(irreps, 6, 8)
    norm = C().LayerNorm(irreps, EPS)
    clean = norm.forward(T(v["x"], dev), T(v["w"], dev), T(v["b"], dev))
    cdx = norm.backward(T(v["x"], dev), T(v["w"], dev), T(v["g"], dev), want=("x",))[0]
    bad = v["x"].copy()
    bad[2, 3], bad[4, 20] = np.nan, np.inf
    y = norm.forward(T(bad, dev), T(v["w"], dev), T(v["b"], dev))
    dx = norm.backward(T(bad, dev), T(v["w"], dev), T(v["g"], dev), want=("x",))[0]
    keep = torch.ones(6, 40, dtype=torch.bool, device=dev)
    keep[2, :16] = False
    keep[4, 16:] = False
    for a, b in ((y, clean), (dx, cdx)):
        assert torch.equal(a[keep], b[keep])
        assert torch.isnan(a[2, :16]).all() and torch.isnan(a[4, 20])


def test_constant_and_zero_rows(dev):
    """Variance zero: r = eps^-1/2, the scalars give the bias, the others 0."""
    norm = C().LayerNorm("8x0e+4x1o", EPS)
    x = torch.zeros(3, 20, device=dev)
    x[1, :8] = 3.0
    b = torch.arange(8.0, device=dev)
    y = norm.forward(x, None, b)
    assert torch.equal(y[:, :8], b.expand(3, 8)) and not y[:, 8:].any()
    g = torch.ones(3, 20, device=dev)
    dx = norm.backward(x, None, g, want=("x",))[0]
    # centred: a - mean(a) = 0; not centred: a / sqrt(eps)
    assert dx[:, :8].abs().max().item() <= K * U / EPS ** 0.5
    assert (dx[:, 8:] - EPS ** -0.5).abs().max().item() <= 8 * U / EPS ** 0.5


def test_repeatable_graph_and_stream(dev):
    """Bitwise the same twice, from another stream, with garbage in workspace
    and outputs, and replayed from two graphs that share one workspace."""
    irreps = "128x0e+64x1o+32x2e"
    v = draw(irreps, 500, 9)
    d = {k: T(a, dev) for k, a in v.items()}
    norm = C().LayerNorm(irreps, EPS)
    ref = (norm.forward(d["x"], d["w"], d["b"]), *norm.backward(d["x"], d["w"], d["g"]),
           *norm.double_backward(d["x"], d["w"], d["g"], d["hx"], d["hw"], d["hb"]))
    ws = torch.full((norm.workspace_size(500),), 255, dtype=torch.uint8, device=dev)
    outs = [torch.full_like(t, float("nan")) for t in ref]

    def first():
        norm.forward(d["x"], d["w"], d["b"], out=outs[0])
        norm.backward(d["x"], d["w"], d["g"], grads=outs[1:4], workspace=ws)

    def second():
        norm.double_backward(d["x"], d["w"], d["g"], d["hx"], d["hw"], d["hb"], grads=outs[4:], workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first()
        second()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    graphs = []
    for f in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for _ in range(2):
        for t in outs:
            t.fill_(float("nan"))
        ws.fill_(255)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_outputs_stay_inside_their_arrays(dev):
    """Guard rows before and behind every output are left as they were."""
    for irreps in ("64x0e", "37x0e+21x1o+11x2e", "1100x0e+340x3o"):
        n = 13
        v = draw(irreps, n, 10)
        d = {k: T(a, dev) for k, a in v.items()}
        norm = C().LayerNorm(irreps, EPS)

        def guarded(m):
            buf = torch.full((m + 128,), 123.0, device=dev)
            return buf, buf[64:64 + m]
        bufs = [guarded(m) for m in (n * norm.d, n * norm.d, norm.n_weight, norm.n_bias, n * norm.d, n * norm.d,
                                     norm.n_weight)]
        o = [b[1] for b in bufs]
        nb = norm.workspace_size(n)
        ws = torch.full((nb + 512,), 77, dtype=torch.uint8, device=dev)
        norm.forward(d["x"], d["w"], d["b"], out=o[0])
        norm.backward(d["x"], d["w"], d["g"], grads=o[1:4], workspace=ws[256:256 + nb])
        norm.double_backward(d["x"], d["w"], d["g"], d["hx"], d["hw"], d["hb"], grads=o[4:], workspace=ws[256:256 + nb])
        torch.cuda.synchronize()
        for buf, t in bufs:
            assert (buf[:64] == 123.0).all() and (buf[64 + t.numel():] == 123.0).all()
        assert (ws[:256] == 77).all() and (ws[256 + nb:] == 77).all()
        assert torch.equal(o[0].view(n, -1), norm.forward(d["x"], d["w"], d["b"]))


def test_gradient_of_the_gradient_by_differences(dev):
    """The second order against differences of the backward on the GPU:
    [S(z + h d) - S(z - h d)] / 2h for a direction d of (g, x, w)."""
    irreps, n = "24x0e+8x1o+4x2e", 40
    v = draw(irreps, n, 11)
    norm = C().LayerNorm(irreps, EPS)
    d = {k: T(a, dev) for k, a in v.items()}
    gg, gx, gw = norm.double_backward(d["x"], d["w"], d["g"], d["hx"], d["hw"], d["hb"])
    rng = np.random.default_rng(12)
    dirs = {k: T(rng.standard_normal(v[k].shape).astype(np.float32), dev) for k in ("g", "x", "w")}

    def S(h):
        a, b, c = norm.backward(d["x"] + h * dirs["x"], d["w"] + h * dirs["w"], d["g"] + h * dirs["g"])
        return sum((p.double() * q.double()).sum().item() for p, q in ((a, d["hx"]), (b, d["hw"]), (c, d["hb"])))
    h = 1e-2
    num = (S(h) - S(-h)) / (2 * h)
    got = sum((p.double() * q.double()).sum().item() for p, q in ((gg, dirs["g"]), (gx, dirs["x"]), (gw, dirs["w"])))
    # truncation h^2 S''' / 6, rounding ~ u sqrt(n D) |S terms| / h: both below 1e-2 of the terms' norm
    scale = sum((p.double() * q.double()).norm().item() for p, q in ((gg, dirs["g"]), (gx, dirs["x"]), (gw, dirs["w"])))
    assert abs(num - got) < 1e-2 * scale


def test_offsets_beyond_32_bits(dev):
    """2.2e9 values an array: the last rows equal the same rows alone."""
    norm = C().LayerNorm("61x0e+1x1o", EPS)
    n = 34_400_001  # x 64 > 2^31
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    tail = torch.randn(4000, 64, device=dev, generator=gen)
    w = torch.randn(62, device=dev, generator=gen)
    x = torch.zeros(n, 64, device=dev)
    x[-4000:] = tail
    y = norm.forward(x, w)
    assert torch.equal(y[-4000:], norm.forward(tail, w))
    del y
    g = torch.zeros(n, 64, device=dev)
    g[-4000:] = 2 * tail
    dx, dw, db = norm.backward(x, w, g)
    rx, rw, rb = norm.backward(tail, w, 2 * tail)
    assert torch.equal(dx[-4000:], rx) and not dx[:1000].any()
    for a, b in ((dw, rw), (db, rb)):  # the same terms, added in another order: 780 u of their magnitudes
        assert (a - b).abs().max().item() <= 2 * (K + 700) * U * 4000 * 64


def test_zero_rows_with_the_smallest_eps(dev):
    eps = float(np.finfo(np.float32).tiny)
    norm = C().LayerNorm("8x0e+4x1o", eps)
    x, g = torch.zeros(3, 20, device=dev), torch.ones(3, 20, device=dev)
    assert not norm.forward(x).any()
    dx, dw, _ = norm.backward(x, None, g)
    assert torch.isfinite(dx).all() and not dw.any()
    assert (dx[:, 8:] * eps ** 0.5 - 1).abs().max().item() <= 8 * U
    gg, gx, gw = norm.double_backward(x, None, g, h_x=g)
    assert torch.isfinite(gg).all() and not gw[:8].any()
