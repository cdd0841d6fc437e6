"""The router's oracle works in FP64 whatever the type of its arguments."""
import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("kw", [dict(renormalise=False), dict(), dict(score="sigmoid"), dict(score="sigmoid", renormalise=False)])
def test_gradients_in_fp32_are_taken_as_they_are(kw):
    """FP32 gradients give the bits that the same values in FP64 give (a product
    with the scale was rounded to FP32)."""
    rng = np.random.default_rng(3)
    l = rng.standard_normal((20, 6)).astype(np.float32)
    ids = O.route_forward(l, None, 3)[0]
    gw, gg = rng.standard_normal((20, 3)).astype(np.float32), rng.standard_normal((6, 20)).astype(np.float32)
    for a, b in ((gw, None), (None, gg), (gw, gg)):
        f = lambda t: None if t is None else t.astype(np.float64)
        got, ref = O.route_backward(l, ids, a, b, scale=1.3, **kw), O.route_backward(l, ids, f(a), f(b), scale=1.3, **kw)
        assert np.array_equal(got, ref)
