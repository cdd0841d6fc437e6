"""GPU parity of the layer norm for rows around and below sqrt(eps), with eps
down to the smallest normal float.

There 1 / sqrt(mean square + eps) is large (9e18 at most) and its powers leave
the range of FP32, though what they are multiplied with brings the results back.
The bounds are those of tests/test_gpu_norm.py, whose inputs and magnitudes are
taken here with rows and cotangents of other sizes.
"""
import numpy as np
import pytest

import oracle as O
import tests.test_gpu_norm as N
from tests.test_gpu_norm import C, K, T, close, dev, draw, magnitudes  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

IRREPS = ["8x0e+4x1o+4x0o", "7x0e+5x1o+3x2e+1x3o", "1100x0e+340x3o", "3x0o+20000x0e+4x1o"]
EPS = [2.0 ** -126, 2.0 ** -100, 2.0 ** -17]


def small(irreps, eps, seed):
    """Rows of 0, 0.1, 1 and 30 times sqrt(eps) (twelve in all, and two of
    size one); grad_y of 30, h_x small enough that nothing exact overflows."""
    v = draw(irreps, 14, seed, offset=0.0)
    rng = np.random.default_rng(seed + 1)
    v["x"] = (rng.standard_normal(v["x"].shape) * (np.array([0, 0.1, 1, 30] * 3 + [0, 0])[:, None] * eps ** 0.5
                                                   + (np.arange(14) >= 12)[:, None])).astype(np.float32)
    v["g"] = (30 * v["g"]).astype(np.float32)
    v["hx"] = (1e-4 * v["hx"]).astype(np.float32)
    return v, {k: T(a, torch.device("cuda:0")) for k, a in v.items()}


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("irreps", IRREPS)
def test_second_order_of_small_rows(irreps, eps, dev, monkeypatch):
    monkeypatch.setattr(N, "EPS", eps)
    v, d = small(irreps, eps, 41)
    mag = magnitudes(irreps, v, 14)
    for keys in (("hx", "hw", "hb"), ("hx",)):
        h = [v[k] if k in keys else np.zeros_like(v[k]) for k in ("hx", "hw", "hb")]
        gg, gx, gw = C().LayerNorm(irreps, eps).double_backward(d["x"], d["w"], d["g"],
                                                                *(d[k] if k in keys else None for k in ("hx", "hw", "hb")))
        rg, rx, rw = O.norm_double_backward(irreps, v["x"], v["w"], v["g"], *h, eps)
        assert np.abs(rx).max() < 1e38
        close(gg, rg, mag["gg"], K, "grad_grad")
        close(gx, rx, mag["gx"], 2 * K, "grad_x")
        close(gw, rw, mag["gw"], K + 700, "grad_weight")


def test_second_order_of_zero_rows(dev):
    """x = 0: gx = r (P k), nothing else; gg = w r P h + h_b; gweight = sum r g P h."""
    eps = float(np.finfo(np.float32).tiny)
    norm = C().LayerNorm("8x0e+4x1o", eps)
    x, g = torch.zeros(3, 20, device=dev), torch.ones(3, 20, device=dev)
    gg, gx, gw = norm.double_backward(x, None, g, h_x=g)
    assert not gx.any() and not gg[:, :8].any() and not gw[:8].any()
    assert (gg[:, 8:] * eps ** 0.5 - 1).abs().max().item() <= 8 * 2.0 ** -24
    assert (gw[8:] * eps ** 0.5 - 9).abs().max().item() <= 9 * 16 * 2.0 ** -24


@pytest.mark.parametrize("eps", EPS)
@pytest.mark.parametrize("irreps", IRREPS)
def test_backward_of_small_rows(irreps, eps, dev, monkeypatch):
    monkeypatch.setattr(N, "EPS", eps)
    v, d = small(irreps, eps, 42)
    mag = magnitudes(irreps, v, 14)
    dx, dw, db = C().LayerNorm(irreps, eps).backward(d["x"], d["w"], d["g"])
    rx, rw, rb = O.norm_backward(irreps, v["x"], v["w"], v["g"], eps)
    close(dx, rx, mag["dx"], K, "grad_x")
    close(dw, rw, mag["dw"], K + 700, "grad_weight")
    close(db, rb, mag["db"], K + 700, "grad_bias")
