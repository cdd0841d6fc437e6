"""One layer of the operators as they are used together (GPU, through the C ABI).

    y = norm(x);  gates = route(logits);  out = sum_b sparse_conv(y, W_b, gates[b])

and its backward: each branch's sparse backward writes its gate gradient into
the row of one array, which the router's backward takes; the branches' dL/dy
add up and go through the norm's backward.  Against the same chain of oracle
functions in FP64 (each pinned on its own) at the acceptance bar of the parity
tests, and against differences of the oracle's forward.  Then the chain that
training on forces differentiates: the convolution's and the norm's double
backward.
"""
import numpy as np
import pytest

import oracle as O
from equivariant_mlip_clebsch_b200 import workloads as WL
from tests._cases import Workload, assert_close

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

EPS = 1e-5
ROUTES = [dict(k=2, score="softmax"), dict(k=1, score="softmax", renormalise=False, scale=1.5),
          dict(k=2, score="sigmoid", n_groups=2, top_groups=1, group_best=1)]


def C():
    from equivariant_mlip_clebsch_b200 import cgtp
    return cgtp


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def T(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


class Layer:
    """Seeded inputs of a layer with n_experts branches on one workload."""

    def __init__(self, name, n_experts, seed=0):
        w = self.w = Workload(name, seed)
        rng = np.random.default_rng([seed, 77])
        f = lambda *s: rng.standard_normal(s).astype(np.float32)
        self.irreps = w.cfg["irreps_in"]
        norm = C().LayerNorm(self.irreps, EPS)
        self.x = (1.5 * w.x + 0.2).astype(np.float32)
        self.weight, self.bias = 1 + 0.2 * f(norm.n_weight), 0.2 * f(norm.n_bias)
        self.W = [WL.normal_f32(w.W.shape, seed + 10 + b, 2, std=w.col_std) for b in range(n_experts)]
        self.logits = f(w.E, n_experts)
        self.logits[rng.random(w.E) < 0.05] = -np.inf  # edges that no branch evaluates
        self.bal = 0.05 * f(n_experts)
        self.Y = O.sph_harm(w.P.L, w.r32)

    def oracle_forward(self, kw, x=None, weight=None, bias=None, logits=None, ids=None):
        """out and what the backward needs; with ids, the choice is held fixed."""
        w = self.w
        pick = lambda a, b: b if a is None else a
        y = O.norm_forward(self.irreps, pick(x, self.x), pick(weight, self.weight), pick(bias, self.bias), EPS)
        if ids is None:
            ids, _, gates, _, _ = O.route_forward(self.logits, self.bal, **kw)
        if logits is not None:  # weights of the fixed choice
            l = np.where(np.isfinite(logits), logits, -1e30)
            e = np.exp(np.minimum(l, 80))
            s = e / np.maximum(e.sum(1, keepdims=True), 1e-300) if kw["score"] == "softmax" else e / (1 + e)
            p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
            if kw.get("renormalise", True):
                p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
            gates = np.zeros((l.shape[1] + 1, len(l)))
            gates[np.where(ids < 0, l.shape[1], ids), np.arange(len(l))[:, None]] = kw.get("scale", 1.0) * p
            gates = gates[:-1]
        out = sum(O.sparse_forward(w.P, w.rowptr, w.col, y, self.Y, Wb, gb) for Wb, gb in zip(self.W, gates))
        return y, ids, gates, out


@pytest.mark.parametrize("kw", ROUTES)
def test_routed_layer_forward_and_backward(kw, dev):
    n_experts = 4
    L = Layer("tiny", n_experts)
    w = L.w
    c = w.cfg
    plan = C().Plan(c["irreps_in"], c["irreps_edge"], c["irreps_out"])
    norm, router = C().LayerNorm(L.irreps, EPS), C().Router(n_experts, **kw)
    rpt, perm = C().csr_transpose(w.rowptr.astype(np.int32), w.col, w.N)
    rowptr, col, rpt, perm = (T(a.astype(np.int32), dev) for a in (w.rowptr, w.col, rpt, perm))
    x, weight, bias, logits, bal, g = (T(a, dev) for a in (L.x, L.weight, L.bias, L.logits, L.bal, w.g))
    W = [T(a, dev) for a in L.W]
    Y = plan.sph_harm(T(w.r32, dev))

    y = norm.forward(x, weight, bias)
    ids, weights, gates, counts = router.forward(logits, bal)
    out = torch.zeros(w.N, plan.d_out, device=dev)
    for b in range(n_experts):
        out += plan.sparse_forward(rowptr, col, y, Y, W[b], gates[b])
    dgates = torch.empty(n_experts, -(-w.E // 4) * 4, device=dev)[:, :w.E]
    dy, dWs = torch.zeros_like(y), []
    for b in range(n_experts):
        grads = (torch.empty_like(y), torch.empty_like(W[b]), None, dgates[b])
        plan.sparse_backward(rowptr, col, rpt, perm, y, Y, W[b], gates[b], g, grads=grads)
        dy += grads[0]
        dWs.append(grads[1])
    dlogits = router.backward(logits, ids, grad_gates=dgates)
    dx, dweight, dbias = norm.backward(x, weight, dy)
    torch.cuda.synchronize()
    plan.check_device_error()

    ry, rids, rgates, rout = L.oracle_forward(kw)
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(rids[rids >= 0], minlength=n_experts))
    rdy, rdg = 0.0, []
    for b in range(n_experts):
        a, rdW, _, d = O.sparse_backward(w.P, w.rowptr, w.col, w.N, ry, L.Y, L.W[b], rgates[b], w.g)
        rdy = rdy + a
        rdg.append(d)
        assert_close(dWs[b].cpu().numpy(), rdW, f"dW of branch {b}")
    rdl = O.route_backward(L.logits, rids, None, np.stack(rdg),
                           **{k: v for k, v in kw.items() if k in ("score", "renormalise", "scale")})
    rdx, rdw, rdb = O.norm_backward(L.irreps, L.x, L.weight, rdy, EPS)
    for name, a, b in (("y", y, ry), ("gates", gates, rgates), ("out", out, rout), ("dgates", dgates, np.stack(rdg)),
                       ("dlogits", dlogits, rdl), ("dx", dx, rdx), ("dweight", dweight, rdw), ("dbias", dbias, rdb)):
        assert_close(a.cpu().numpy(), b, name)

    # along one direction of every input, the loss's difference quotient (FP64, the choice held fixed)
    rng = np.random.default_rng(5)
    d = {k: rng.standard_normal(v.shape) for k, v in (("x", L.x), ("weight", L.weight), ("bias", L.bias),
                                                      ("logits", L.logits))}
    h = 1e-5
    loss = lambda s: float((L.oracle_forward(kw, *(v + s * h * d[k] for k, v in (
        ("x", L.x.astype(np.float64)), ("weight", L.weight), ("bias", L.bias), ("logits", L.logits))),
        ids=rids)[3] * w.g).sum())
    num = (loss(1) - loss(-1)) / (2 * h)
    parts = [(a.double().cpu().numpy() * np.where(np.isfinite(d[k]), d[k], 0)).sum()
             for a, k in ((dx, "x"), (dweight, "weight"), (dbias, "bias"), (dlogits, "logits"))]
    # FP32 gradients at the bar's 1e-5 of their norm each; the quotient's truncation is h^2
    scale = sum(float(a.double().norm()) * np.linalg.norm(d[k]) for a, k in (
        (dx, "x"), (dweight, "weight"), (dbias, "bias"), (dlogits, "logits")))
    assert abs(sum(parts) - num) <= 1e-5 * scale


def test_routed_layer_in_one_graph(dev):
    """The whole step captured once and replayed: bit for bit the eager one."""
    kw, n_experts = ROUTES[0], 4
    L = Layer("tiny", n_experts)
    w, c = L.w, L.w.cfg
    plan = C().Plan(c["irreps_in"], c["irreps_edge"], c["irreps_out"])
    norm, router = C().LayerNorm(L.irreps, EPS), C().Router(n_experts, **kw)
    rpt, perm = C().csr_transpose(w.rowptr.astype(np.int32), w.col, w.N)
    rowptr, col, rpt, perm = (T(a.astype(np.int32), dev) for a in (w.rowptr, w.col, rpt, perm))
    x, weight, bias, logits, bal, g = (T(a, dev) for a in (L.x, L.weight, L.bias, L.logits, L.bal, w.g))
    W = [T(a, dev) for a in L.W]
    Y = plan.sph_harm(T(w.r32, dev))

    def step():
        y = norm.forward(x, weight, bias)
        ids, _, gates, _ = router.forward(logits, bal)
        dgates = torch.empty(n_experts, -(-w.E // 4) * 4, device=dev)[:, :w.E]
        outs, dy = [], torch.zeros_like(y)
        for b in range(n_experts):
            outs.append(plan.sparse_forward(rowptr, col, y, Y, W[b], gates[b]))
            dyb, _, _, dg = plan.sparse_backward(rowptr, col, rpt, perm, y, Y, W[b], gates[b], g, want=("x", "gate"))
            dy += dyb
            dgates[b].copy_(dg)
        return (*outs, router.backward(logits, ids, grad_gates=dgates), *norm.backward(x, weight, dy))
    eager = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


@pytest.mark.parametrize("name", ["tiny", "lmax2"])
def test_norm_and_convolution_double_backward(name, dev):
    """S = <h, dE/dx> of E = <g, conv(norm(x))>, as a loss on forces uses it:
    dS/dg = conv(J h'), dS/dx and dS/dweight through the norm's double backward
    with the convolution's gradient as its cotangent."""
    w = Workload(name)
    c = w.cfg
    irreps = c["irreps_in"]
    rng = np.random.default_rng(9)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    plan, norm = C().Plan(c["irreps_in"], c["irreps_edge"], c["irreps_out"]), C().LayerNorm(irreps, EPS)
    weight, bias, h = 1 + 0.2 * f(norm.n_weight), f(norm.n_bias), f(*w.x.shape)
    rpt, perm = C().csr_transpose(w.rowptr.astype(np.int32), w.col, w.N)
    rowptr, col, rpt, perm = (T(a.astype(np.int32), dev) for a in (w.rowptr, w.col, rpt, perm))
    Yd, Wd, gd, xd = plan.sph_harm(T(w.r32, dev)), T(w.W, dev), T(w.g, dev), T(w.x, dev)
    y = norm.forward(xd, T(weight, dev), T(bias, dev))
    gy, _, _ = plan.backward(rowptr, col, rpt, perm, y, Yd, Wd, gd, want=("x",))
    hy, gx, gw = norm.double_backward(xd, T(weight, dev), gy, h_x=T(h, dev))
    gg, _, cW, cY = plan.double_backward(rowptr, col, rpt, perm, y, Yd, Wd, gd, h_x=hy, want=("g", "W", "Y"))
    torch.cuda.synchronize()
    plan.check_device_error()
    Y = O.sph_harm(w.P.L, w.r32)
    ry = O.norm_forward(irreps, w.x, weight, bias, EPS)
    rgy = O.backward(w.P, w.rowptr, w.col, w.N, ry, Y, w.W, w.g, want=("x",))[0]
    rhy, rgx, rgw = O.norm_double_backward(irreps, w.x, weight, rgy, h, np.zeros_like(weight), np.zeros_like(bias), EPS)
    rgg = O.forward(w.P, w.rowptr, w.col, rhy, Y, w.W)
    _, rcW, rcY = O.backward(w.P, w.rowptr, w.col, w.N, rhy, Y, w.W, w.g)
    for what, a, b in (("gy", gy, rgy), ("hy", hy, rhy), ("gx", gx, rgx), ("gweight", gw, rgw), ("dS/dg", gg, rgg),
                       ("dS/dW", cW, rcW), ("dS/dY", cY, rcY)):
        assert_close(a.cpu().numpy(), b, what)
