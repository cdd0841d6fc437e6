"""The layer norm over irreps rows and the router of edges to experts: cases, inputs, plain forms.

Operators (the field ``op`` of a case):
  norm_forward, norm_backward, norm_double_backward
      rows of irreps blocks "MxLp+...", each block [mul, 2l+1]; every block of a row is normalised by itself:
      0e blocks are centred and have a weight and a bias a channel, the others are divided by their root mean
      square and have a weight a channel.  "64x0e" is the plain layer norm of 64 columns.
  route_forward, route_backward
      scores of n experts an edge, the k best chosen (with a bias, and within the best groups), their weights,
      and the gates [expert, edge] that the convolution's sparse evaluation takes.

``own`` is set from outside: False runs the plain torch forms, True the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
LOWEST = torch.finfo(torch.float32).min

LMAX3_IN = "128x0e+64x1o+32x2e+32x3o"
LMAX3_OUT = "256x0e+352x1o+384x2e+320x3o"
LMAX6_OUT = "448x0e+768x1o+1024x2e+1152x3o+1216x4e+1152x5o+1024x6e"


def listed():
    return [
        # the smallest workload's node features: 64 atoms, one launch's latency
        dict(name="norm_fwd tiny", op="norm_forward", rows=64, irreps="16x0e+16x1o"),
        # hidden features between two convolutions, 6,144 atoms, Lmax 3
        dict(name="norm_fwd lmax3 hidden", op="norm_forward", rows=6144, irreps=LMAX3_IN),
        # the widest convolution output, Lmax 6: 52,864 floats an atom
        dict(name="norm_fwd lmax6 out", op="norm_forward", rows=768, irreps=LMAX6_OUT),
        # training on 768 atoms, Lmax 2 hidden features
        dict(name="norm_bwd lmax2 hidden", op="norm_backward", rows=768, irreps="128x0e+64x1e+32x2e"),
        # the plain layer norm of an edge network's 64 hidden columns; many short rows, an odd number
        dict(name="norm_bwd edge scalars", op="norm_backward", rows=172051, irreps="64x0e"),
        # training through the norm of a convolution's output, the largest case
        dict(name="norm_bwd lmax3 out", op="norm_backward", rows=6144, irreps=LMAX3_OUT),
        # odd multiplicities: rows that start on no 16-byte border
        dict(name="norm_dbwd odd", op="norm_double_backward", rows=1001, irreps="37x0e+21x1o+11x2e"),
        # training on forces, 6,144 atoms, Lmax 3 hidden features
        dict(name="norm_dbwd lmax3 hidden", op="norm_double_backward", rows=6144, irreps=LMAX3_IN),
        # 1,792 edges of the smallest workload over four branches
        dict(name="route_fwd tiny", op="route_forward", rows=1792, experts=4, k=1, score="softmax", groups=1,
             top_groups=1, group_best=1, renormalise=False, scale=1.0, bias=False, masked=False),
        # every edge of 6,144 atoms over 64 experts in groups, balanced by a bias; some edges and experts masked
        dict(name="route_fwd grouped", op="route_forward", rows=172050, experts=64, k=8, score="sigmoid", groups=8,
             top_groups=4, group_best=2, renormalise=True, scale=2.5, bias=True, masked=True),
        # gradient of plain softmax gates: every expert's logit gets one
        dict(name="route_bwd softmax", op="route_backward", rows=34244, experts=16, k=2, score="softmax", groups=1,
             top_groups=1, group_best=1, renormalise=False, scale=1.0, bias=False, masked=False),
        # gradient of the grouped router above
        dict(name="route_bwd grouped", op="route_backward", rows=172050, experts=64, k=8, score="sigmoid", groups=8,
             top_groups=4, group_best=2, renormalise=True, scale=2.5, bias=True, masked=True),
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: any operator, one row up to the listed sizes, odd sizes among them."""
    op = rng.choice(["norm_forward", "norm_backward", "norm_double_backward", "route_forward", "route_backward"])
    if op.startswith("norm"):
        blocks, l = [], rng.choice([0, 0, 0, 1])
        for _ in range(rng.randint(1, 5)):
            if l > 6:
                break
            mul = _log(rng, 4 if l == 0 else 1, 1024 // (l + 1))  # two scalars or one: the gradient is all rounding
            if rng.random() < 0.5:
                mul = -(-mul // 4) * 4
            blocks.append("%dx%d%s" % (mul, l, rng.choice("eeo") if l == 0 else rng.choice("eo")))
            l += rng.choice([1, 1, 2]) if rng.random() < 0.85 else 0
        irreps = "+".join(blocks)
        width = sum(m * (2 * l + 1) for m, l, _ in _blocks(irreps))
        streams = {"norm_forward": 2, "norm_backward": 3, "norm_double_backward": 5}[op]
        most = max(1, min(200000, int(9e7 / streams / width)))
        return dict(op=op, rows=_log(rng, 1, most), irreps=irreps)
    n = _log(rng, 2, 256)
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if n % g == 0])
    top = rng.randint(1, groups)
    k = rng.randint(1, min(8, n // groups * top))
    rows = _log(rng, 1, max(1, min(200000, 11000000 // n)))
    return dict(op=op, rows=rows, experts=n, k=k, score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                top_groups=top, group_best=rng.choice([1, 2]), renormalise=rng.random() < 0.6,
                scale=rng.choice([1.0, 1.0, 2.5]), bias=rng.random() < 0.6, masked=rng.random() < 0.5)


def _blocks(irreps):
    """[(mul, l, parity letter)] of an irreps string."""
    got = []
    for t in irreps.split("+"):
        mul, rest = t.split("x")
        got.append((int(mul), int(rest[:-1]), rest[-1]))
    return got


def _layout(irreps, device):
    """For every column of a row: its block and its channel; for every block: its length and whether it is centred;
    the channels that have a bias."""
    blocks = _blocks(irreps)
    size = np.array([m * (2 * l + 1) for m, l, _ in blocks])
    seg = np.repeat(np.arange(len(blocks)), size)
    muls, degree = [m for m, _, _ in blocks], [2 * l + 1 for _, l, _ in blocks]
    channel = np.repeat(np.arange(sum(muls)), np.repeat(degree, muls))
    scalar = np.array([l == 0 and p == "e" for _, l, p in blocks])
    biased = np.flatnonzero(np.repeat(scalar, muls))
    t = lambda a, d=None: torch.from_numpy(np.ascontiguousarray(a)).to(device, d)  # noqa: E731
    member = (seg[:, None] == np.arange(len(blocks))[None, :]).astype(np.float32)  # [D, blocks]
    return dict(seg=t(seg), channel=t(channel), mean=t(member / size[None, :].astype(np.float32), torch.float32),
                centred=t(scalar.astype(np.float32)), biased=t(biased), channels=int(channel[-1]) + 1,
                cols=t(np.flatnonzero(scalar[seg])))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    normal = lambda *s: torch.randn(s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    uniform = lambda *s: torch.rand(s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    n = case["rows"]
    if case["op"].startswith("norm"):
        lay = _layout(case["irreps"], dev)
        D, C, B = lay["seg"].numel(), lay["channels"], lay["biased"].numel()
        s = dict(case=case, lay=lay)
        # features as a convolution leaves them: every row of its own size, an offset on every column
        s["x"] = normal(n, D) * torch.exp(0.5 * normal(n, 1)) + 0.3 * normal(1, D)
        s["weight"] = 1 + 0.2 * normal(C)
        s["bias"] = 0.2 * normal(B)
        if case["op"] != "norm_forward":
            s["grad"] = normal(n, D)
        if case["op"] == "norm_double_backward":
            s["h_x"], s["h_weight"], s["h_bias"] = normal(n, D), 0.1 * normal(C), 0.1 * normal(B)
    else:
        E, k = case["experts"], case["k"]
        s = dict(case=case)
        s["logits"] = 1.5 * normal(n, E) + 0.5 * normal(1, E)
        if case["masked"]:  # single experts out for an edge, and edges (padding) with none left
            s["logits"].masked_fill_(uniform(n, E) < 0.03, -math.inf)
            s["logits"].masked_fill_(uniform(n, 1) < 0.02, LOWEST)
        s["bias"] = 0.05 * normal(E) if case["bias"] else None
        if case["op"] == "route_backward":
            s["ids"] = _select(case, *_scores(case, s["logits"], s["bias"])).to(torch.int32)
            # the convolution's gradient of the gates: zero where an edge was not evaluated
            ld = -(-n // 4) * 4
            chosen = torch.zeros(n, E + 1, device=dev).scatter_(1, torch.where(s["ids"] < 0, E, s["ids"]).long(), 1.0)
            s["grad_gates"] = torch.zeros(E, ld, device=dev)[:, :n]
            s["grad_gates"].copy_((normal(n, E) * chosen[:, :E]).t())
    if own:
        from equivariant_mlip_clebsch_b200 import cgtp
        if case["op"].startswith("norm"):
            s["norm"] = cgtp.LayerNorm(case["irreps"], EPS)
            if case["op"] != "norm_forward":
                s["workspace"] = torch.empty(max(s["norm"].workspace_size(n), 256), dtype=torch.uint8, device=dev)
        else:
            s["router"] = cgtp.Router(case["experts"], case["k"], score=case["score"], n_groups=case["groups"],
                                      top_groups=case["top_groups"], group_best=case["group_best"],
                                      renormalise=case["renormalise"], scale=case["scale"])
    return s


def run(s):
    op = s["case"]["op"]
    return (_run_own if own else _run_plain)(op, s)


def _run_own(op, s):
    if op == "norm_forward":
        return {"y": s["norm"].forward(s["x"], s["weight"], s["bias"])}
    if op == "norm_backward":
        dx, dw, db = s["norm"].backward(s["x"], s["weight"], s["grad"], workspace=s["workspace"])
        return {"grad_x": dx, "grad_weight": dw, "grad_bias": db}
    if op == "norm_double_backward":
        gg, gx, gw = s["norm"].double_backward(s["x"], s["weight"], s["grad"], h_x=s["h_x"], h_weight=s["h_weight"],
                                               h_bias=s["h_bias"], workspace=s["workspace"])
        return {"grad_grad": gg, "grad_x": gx, "grad_weight": gw}
    if op == "route_forward":
        ids, weights, gates, counts = s["router"].forward(s["logits"], s["bias"])
        return {"ids": ids, "weights": weights, "gates": gates, "counts": counts}
    return {"grad_logits": s["router"].backward(s["logits"], s["ids"], grad_gates=s["grad_gates"])}


# ---- plain forms


def _run_plain(op, s):
    if op.startswith("norm"):
        return _norm_plain(op, s)
    if op == "route_forward":
        return _route_plain(s)
    return _route_backward_plain(s)


def _norm_plain(op, s):
    lay = s["lay"]
    seg, channel, centred = lay["seg"], lay["channel"], lay["centred"]
    x, w = s["x"], s["weight"][channel]
    mean = lambda z: z @ lay["mean"]  # of every block: [N, blocks]  # noqa: E731
    centre = lambda z: z - (mean(z) * centred)[:, seg]  # noqa: E731
    xc = centre(x)
    r = torch.rsqrt(mean(xc * xc) + EPS)[:, seg]
    xh = xc * r
    if op == "norm_forward":
        y = xh * w
        shift = torch.zeros(lay["channels"], device=x.device).index_copy_(0, lay["biased"], s["bias"])[channel]
        return {"y": y + shift}
    to_channels = lambda v: torch.zeros(lay["channels"], device=x.device).index_add_(0, channel, v)  # noqa: E731
    g = s["grad"]
    a = w * g
    if op == "norm_backward":
        gx = r * (centre(a) - xh * mean(a * xh)[:, seg])
        return {"grad_x": gx, "grad_weight": to_channels((g * xh).sum(0)), "grad_bias": g.sum(0)[lay["cols"]]}
    h, c = s["h_x"], s["h_weight"][channel] * g
    pa, ph = centre(a), centre(h)
    al, be, ga = mean(a * xh)[:, seg], mean(h * xh)[:, seg], mean(ph * a)[:, seg]
    jh = r * (ph - xh * be)
    shift = torch.zeros(lay["channels"], device=x.device).index_copy_(0, lay["biased"], s["h_bias"])[channel]
    gg = w * jh + s["h_weight"][channel] * xh + shift
    gx = r * r * (xh * (3 * al * be - ga) - be * pa - al * ph) + r * (centre(c) - xh * mean(c * xh)[:, seg])
    return {"grad_grad": gg, "grad_x": gx, "grad_weight": to_channels((g * jh).sum(0))}


def _scores(case, logits, bias):
    """Scores (0 where an expert is out), and the biased scores that are compared (-inf there), in 64 bits: the
    choice goes by values that may be next to one another."""
    l = logits.double()
    there = logits > LOWEST
    if case["score"] == "softmax":
        top = torch.where(there, l, -math.inf).amax(1, keepdim=True)
        e = torch.where(there, torch.exp(l - torch.where(torch.isfinite(top), top, 0.0)), 0.0)
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total > 0, total, 1.0)
    else:
        score = torch.where(there, 1 / (1 + torch.exp(-l)), 0.0)
    biased = score if bias is None else score + bias.double()
    return score, torch.where(there, biased, -math.inf)


def _select(case, score, biased):
    """The chosen experts of every row, best first, the lowest index first where two are equal; -1 where none is left."""
    n, E = biased.shape
    G, k = case["groups"], case["k"]
    if G > 1:
        each = biased.view(n, G, E // G)
        best = each.sort(dim=-1, descending=True).values[..., : min(case["group_best"], E // G)]
        total = torch.where(torch.isfinite(best), best, 0.0).sum(-1)
        total = torch.where(torch.isfinite(best[..., 0]), total, -math.inf)
        order = total.sort(dim=-1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros(n, G, dtype=torch.bool, device=biased.device).scatter_(1, order, True)
        biased = torch.where(keep[:, :, None], each, -math.inf).reshape(n, E)
    v, i = biased.sort(dim=-1, descending=True, stable=True)
    return torch.where(v[:, :k] > -math.inf, i[:, :k], -1)


def _weights(case, score, ids):
    """Weights of the chosen experts from the scores, in the scores' type."""
    p = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalise"]:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    return case["scale"] * p


def _route_plain(s):
    case, E = s["case"], s["case"]["experts"]
    score, biased = _scores(case, s["logits"], s["bias"])
    ids = _select(case, score, biased)
    weights = _weights(case, score, ids).float()
    slot = torch.where(ids >= 0, ids, E)
    gates = torch.zeros(ids.shape[0], E + 1, device=ids.device).scatter_(1, slot, weights)[:, :E].t()
    chosen = torch.zeros(ids.shape[0], E + 1, dtype=torch.int32, device=ids.device).scatter_(1, slot, 1)[:, :E]
    counts = chosen.sum(0, dtype=torch.int32)
    return {"ids": ids.to(torch.int32), "weights": weights, "gates": gates.contiguous(), "counts": counts}


def _route_backward_plain(s):
    case, ids = s["case"], s["ids"].long()
    l = s["logits"]
    there = l > LOWEST
    E, scale = case["experts"], case["scale"]
    held, row = ids >= 0, ids.clamp(min=0)
    dw = torch.where(held, s["grad_gates"].t().gather(1, row), 0.0)
    soft = case["score"] == "softmax"
    if soft:
        top = torch.where(there, l, LOWEST).amax(1, keepdim=True)
        e = torch.where(there, torch.exp(l - top), 0.0)
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total > 0, total, 1.0)
    else:
        score = torch.where(there, 1 / (1 + torch.exp(-l)), 0.0)
    p = torch.where(held, score.gather(1, row), 0.0)
    if case["renormalise"]:
        total = p.sum(1, keepdim=True)
        q = p / torch.where(total > 0, total, 1.0)  # = weight / scale
        d = scale * q * (dw - (dw * q).sum(1, keepdim=True))
        d = d if soft else d * (1 - p)
    else:
        d = scale * dw * p * (1 if soft else 1 - p)
    slot = torch.where(held, ids, E)
    out = torch.zeros(ids.shape[0], E + 1, device=l.device).scatter_(1, slot, d)[:, :E]
    if soft and not case["renormalise"]:
        out = out - score * d.sum(1, keepdim=True)
    return {"grad_logits": out.contiguous()}


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    n = case["rows"]
    if case["op"].startswith("norm"):
        blocks = _blocks(case["irreps"])
        D = sum(m * (2 * l + 1) for m, l, _ in blocks)
        C, B = sum(m for m, _, _ in blocks), sum(m for m, l, p in blocks if l == 0 and p == "e")
        streams, params, ops = {"norm_forward": (2, C + B, 8), "norm_backward": (3, 2 * C + B, 16),
                                "norm_double_backward": (5, 3 * C + B, 35)}[case["op"]]
        return {"bytes": 4 * (streams * n * D + params), "flops": ops * n * D}
    E, k = case["experts"], case["k"]
    if case["op"] == "route_forward":
        return {"bytes": 4 * (n * E + (E if case["bias"] else 0) + 2 * n * k + n * E + E), "flops": 12 * n * E}
    every = case["score"] == "softmax" and not case["renormalise"]  # else only the chosen experts' logits count
    return {"bytes": 4 * (n * (E if every else k) + 2 * n * k + n * E), "flops": n * (6 * E if every else 12 * k)}


# ---- the definition in 64 bits


def _norm64(irreps, x, w, b):
    """The forward by blocks, in the type of its arguments (64 bits)."""
    got, col, ch, sc = [], 0, 0, 0
    for mul, l, p in _blocks(irreps):
        d = 2 * l + 1
        z = x[:, col:col + mul * d].reshape(-1, mul, d)
        if l == 0 and p == "e":
            z = z - z.mean(dim=(1, 2), keepdim=True)
        z = z / torch.sqrt((z ** 2).mean(dim=(1, 2), keepdim=True) + EPS) * w[None, ch:ch + mul, None]
        if l == 0 and p == "e":
            z = z + b[None, sc:sc + mul, None]
            sc += mul
        got.append(z.reshape(x.shape[0], mul * d))
        col, ch = col + mul * d, ch + mul
    return torch.cat(got, dim=1)


def _route64(case, logits, bias):
    """ids, weights by a loop over the choices, numpy in 64 bits."""
    l = logits.astype(np.float64)
    out = ~(logits > LOWEST)
    n, E = l.shape
    lm = np.where(out, -np.inf, l)
    if case["score"] == "softmax":
        top = lm.max(1, keepdims=True)
        e = np.exp(lm - np.where(np.isfinite(top), top, 0.0))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    else:
        s = 1.0 / (1.0 + np.exp(-np.where(out, 0.0, l)))
        s[out] = 0.0
    v = s.copy() if bias is None else s + bias.astype(np.float64)[None]
    v[out] = -np.inf
    if case["groups"] > 1:
        size = E // case["groups"]
        total = np.full((n, case["groups"]), -np.inf)
        for j in range(case["groups"]):
            part = -np.sort(-v[:, j * size:(j + 1) * size], axis=1)[:, :case["group_best"]]
            total[:, j] = np.where(np.isfinite(part[:, 0]), np.where(np.isfinite(part), part, 0.0).sum(1), -np.inf)
        rank = np.argsort(np.argsort(-total, axis=1, kind="stable"), axis=1, kind="stable")
        v[np.repeat(rank >= case["top_groups"], size, axis=1)] = -np.inf
    ids, rows = np.full((n, case["k"]), -1, dtype=np.int64), np.arange(n)
    for j in range(case["k"]):
        at = v.argmax(1)  # the first of equal ones
        ids[:, j] = np.where(v[rows, at] > -np.inf, at, -1)
        v[rows, at] = -np.inf
    p = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if case["renormalise"]:
        p = p / np.maximum(p.sum(1, keepdims=True), 1e-300)
    return ids, case["scale"] * p


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        up = lambda k: s[k].double().requires_grad_(True)  # noqa: E731
        x, w, b = up("x"), up("weight"), up("bias")
        if case["op"] == "norm_forward":
            return {"y": _norm64(case["irreps"], x, w, b).detach()}
        g = up("grad")
        y = _norm64(case["irreps"], x, w, b)
        if case["op"] == "norm_backward":
            dx, dw, db = torch.autograd.grad(y, (x, w, b), g, allow_unused=True)
            return {"grad_x": dx, "grad_weight": dw, "grad_bias": torch.zeros_like(b) if db is None else db}
        dx, dw, db = torch.autograd.grad(y, (x, w, b), g, create_graph=True, allow_unused=True)
        S = (dx * s["h_x"].double()).sum() + (dw * s["h_weight"].double()).sum()
        if db is not None:
            S = S + (db * s["h_bias"].double()).sum()
        gg, gx, gw = torch.autograd.grad(S, (g, x, w))
        return {"grad_grad": gg, "grad_x": gx, "grad_weight": gw}
    E, n = case["experts"], case["rows"]
    logits = s["logits"].cpu().numpy()
    rows = np.arange(n)[:, None]
    if case["op"] == "route_forward":
        ids, w = _route64(case, logits, None if s["bias"] is None else s["bias"].cpu().numpy())
        gates = np.zeros((n, E + 1))
        gates[rows, np.where(ids < 0, E, ids)] = w
        return {"ids": ids, "weights": w, "gates": np.ascontiguousarray(gates[:, :E].T),
                "counts": np.bincount(ids[ids >= 0].ravel(), minlength=E)}
    # the gradient through the weights of the given choice, by torch's differentiation in 64 bits
    l = s["logits"].double().requires_grad_(True)
    there = s["logits"] > LOWEST
    if case["score"] == "softmax":
        some = there.any(1, keepdim=True)
        score = torch.softmax(torch.where(there, l, torch.where(some, -math.inf, 0.0).double()), 1) * there
    else:
        score = torch.sigmoid(torch.where(there, l, 0.0)) * there
    ids = s["ids"].long()
    held = ids >= 0
    p = torch.where(held, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalise"]:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    dw = torch.where(held, s["grad_gates"].double().t().gather(1, ids.clamp(min=0)), 0.0)
    (dl,) = torch.autograd.grad((case["scale"] * p * dw).sum(), l)
    return {"grad_logits": dl}
