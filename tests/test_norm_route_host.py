"""Refusals of the layer norm and the router (no GPU needed): every call is
refused before any launch, by the C ABI or by the binding."""
import ctypes

import pytest

from equivariant_mlip_clebsch_b200 import cgtp as C

OK, NULL, ALIGN, PARSE, LMAX, SIZE, WORKSPACE = 0, 1, 2, 3, 5, 6, 12
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("irreps,eps,status", [
    ("16x0e+", 1e-5, PARSE), ("", 1e-5, PARSE), ("0x0e", 1e-5, PARSE), ("16x7e", 1e-5, LMAX),
    ("16x0e", 0.0, SIZE), ("16x0e", -1.0, SIZE), ("16x0e", float("nan"), SIZE), ("16x0e", float("inf"), SIZE),
    ("16x0e", 1e-60, SIZE), ("16x0e", 1e-40, SIZE), ("16x0e", 1e39, SIZE), ("+".join(["2x0e"] * 33), 1e-5, SIZE),
    ("+".join(["1000000x6e"] * 32) + "+8x0e", 1e-5, SIZE), ("+".join(["1048576x6e"] * 32), 1e-5, OK),
])
def test_norm_create_refusals(irreps, eps, status):
    if status == OK:  # 32 blocks of the largest multiplicity stay below 2^30 columns
        assert C.LayerNorm(irreps, eps).d == 32 * 1048576 * 13
        return
    with pytest.raises(C.CgtpError) as e:
        C.LayerNorm(irreps, eps)
    assert e.value.status == status


def test_norm_info():
    n = C.LayerNorm("5x0e+3x1o+2x0o+4x0e")
    assert (n.d, n.n_weight, n.n_bias) == (20, 14, 9)
    assert C.LayerNorm("+".join(["2x0e"] * 32)).d == 64


def test_norm_abi_refusals():
    lib = C._lib
    n = C.LayerNorm("8x0e+4x1o")
    p, odd = ctypes.c_void_p(256), ctypes.c_void_p(260)  # never dereferenced: refused first
    assert lib.cgtp_norm_create(b"8x0e", 1e-5, None) == NULL
    h = ctypes.c_void_p(1)
    assert lib.cgtp_norm_create(None, 1e-5, ctypes.byref(h)) == NULL and not h.value
    assert lib.cgtp_norm_destroy(None) == OK
    assert lib.cgtp_norm_info(None, None, None, None) == NULL
    assert lib.cgtp_norm_info(n._h, None, None, None) == OK
    f = lib.cgtp_norm_forward
    assert f(None, 1, p, p, p, p, None) == NULL
    assert f(n._h, -1, p, p, p, p, None) == SIZE
    assert f(n._h, 1 << 31, p, p, p, p, None) == SIZE
    assert f(n._h, 0, None, None, None, None, None) == OK
    assert f(n._h, 3, None, p, p, p, None) == NULL
    assert f(n._h, 3, p, p, p, None, None) == NULL
    for k in range(4):
        assert f(n._h, 3, *[odd if j == k else p for j in range(4)], None) == ALIGN
    size = ctypes.c_size_t()
    assert lib.cgtp_norm_workspace_size(n._h, -1, ctypes.byref(size)) == SIZE
    assert lib.cgtp_norm_workspace_size(n._h, 5, None) == NULL
    assert lib.cgtp_norm_workspace_size(n._h, 5, ctypes.byref(size)) == OK and size.value > 0
    b = lib.cgtp_norm_backward
    assert b(None, 3, p, p, p, p, p, p, p, 1 << 30, None) == NULL
    assert b(n._h, 3, None, p, p, p, p, p, p, 1 << 30, None) == NULL
    assert b(n._h, 3, p, p, None, p, p, p, p, 1 << 30, None) == NULL
    assert b(n._h, 3, p, p, p, p, p, p, None, 0, None) == WORKSPACE
    assert b(n._h, 3, p, p, p, p, p, p, p, size.value * 0, None) == WORKSPACE
    assert b(n._h, 3, p, p, p, p, p, p, odd, 1 << 30, None) == ALIGN
    for k in range(6):
        assert b(n._h, 3, *[odd if j == k else p for j in range(6)], p, 1 << 30, None) == ALIGN
    assert b(n._h, 3, p, p, p, None, None, None, None, 0, None) == OK  # nothing asked for
    d = lib.cgtp_norm_double_backward
    assert d(None, 3, *[p] * 10, 1 << 30, None) == NULL
    assert d(n._h, 3, None, *[p] * 9, 1 << 30, None) == NULL
    assert d(n._h, 3, p, p, None, *[p] * 7, 1 << 30, None) == NULL
    assert d(n._h, 3, *[p] * 9, None, 0, None) == WORKSPACE
    for k in range(9):
        assert d(n._h, 3, *[odd if j == k else p for j in range(9)], p, 1 << 30, None) == ALIGN
    assert d(n._h, 3, p, p, p, p, p, p, None, None, None, None, 0, None) == OK


@pytest.mark.parametrize("kw", [
    dict(n_experts=0, k=1), dict(n_experts=513, k=1), dict(n_experts=8, k=0), dict(n_experts=8, k=9),
    dict(n_experts=64, k=33), dict(n_experts=8, k=1, n_groups=3), dict(n_experts=8, k=1, n_groups=0),
    dict(n_experts=64, k=1, n_groups=64), dict(n_experts=8, k=1, n_groups=4, top_groups=5),
    dict(n_experts=8, k=1, n_groups=4, top_groups=0), dict(n_experts=8, k=5, n_groups=4, top_groups=2),
    dict(n_experts=8, k=1, group_best=3), dict(n_experts=8, k=1, scale=0.0),
    dict(n_experts=8, k=1, scale=float("inf")), dict(n_experts=8, k=1, scale=float("nan")),
])
def test_router_create_refusals(kw):
    with pytest.raises(C.CgtpError) as e:
        C.Router(**kw)
    assert e.value.status == SIZE


def test_router_limits_are_accepted():
    for kw in (dict(n_experts=512, k=32), dict(n_experts=1, k=1), dict(n_experts=64, k=8, n_groups=32, top_groups=4)):
        assert C.Router(**kw).k == kw["k"]
    with pytest.raises(ValueError, match="score"):
        C.Router(8, 2, score="relu")


def test_router_abi_refusals():
    lib = C._lib
    r = C.Router(8, 2)
    p, odd = ctypes.c_void_p(256), ctypes.c_void_p(260)
    assert lib.cgtp_router_create(8, 2, 7, 1, 1, 1, 1, 1.0, ctypes.byref(ctypes.c_void_p())) == SIZE
    assert lib.cgtp_router_create(8, 2, 0, 1, 1, 1, 1, 1.0, None) == NULL
    assert lib.cgtp_router_destroy(None) == OK
    f = lib.cgtp_router_forward
    assert f(None, 3, p, p, p, p, p, 4, p, None) == NULL
    assert f(r._h, -1, p, p, p, p, p, 4, p, None) == SIZE
    assert f(r._h, 1 << 31, p, p, p, p, p, 1 << 31, p, None) == SIZE
    assert f(r._h, 5, p, p, p, p, p, 4, p, None) == SIZE  # rows of gates overlap
    assert f(r._h, 5, p, p, p, p, p, 6, p, None) == SIZE  # not a multiple of 4
    assert f(r._h, 5, None, p, p, p, p, 8, p, None) == NULL
    for k in range(5):
        assert f(r._h, 5, *[odd if j == k else p for j in range(5)], 8, p, None) == ALIGN
    assert f(r._h, 5, p, p, p, p, p, 8, odd, None) == ALIGN
    assert f(r._h, 5, p, p, None, None, None, 0, None, None) == OK  # nothing asked for
    assert f(r._h, 0, None, None, None, None, None, 0, None, None) == OK
    b = lib.cgtp_router_backward
    assert b(None, 5, p, p, p, p, 8, p, None) == NULL
    assert b(r._h, -1, p, p, p, p, 8, p, None) == SIZE
    assert b(r._h, 5, p, p, p, p, 4, p, None) == SIZE
    assert b(r._h, 5, None, p, p, p, 8, p, None) == NULL
    assert b(r._h, 5, p, None, p, p, 8, p, None) == NULL
    assert b(r._h, 5, p, p, p, p, 8, None, None) == NULL
    assert b(r._h, 0, None, None, None, None, 0, None, None) == OK
    for k in range(4):
        assert b(r._h, 5, *[odd if j == k else p for j in range(4)], 8, p, None) == ALIGN
    assert b(r._h, 5, p, p, p, p, 8, odd, None) == ALIGN


def test_binding_checks_tensors():
    n = C.LayerNorm("8x0e+4x1o")
    x, w, b = torch.zeros(3, 20), torch.ones(12), torch.zeros(8)
    with pytest.raises(TypeError, match="x: expected torch.float32"):
        n.forward(x.double(), w, b)
    with pytest.raises(TypeError, match="weight: expected torch.float32"):
        n.forward(x, w.half(), b)
    with pytest.raises(ValueError, match="x: expected 60 elements"):
        n.forward(x[:, :19].contiguous(), w, b)
    with pytest.raises(ValueError, match="bias: expected 8 elements"):
        n.forward(x, w, w)
    with pytest.raises(ValueError, match="out: expected"):
        n.forward(x, w, b, out=x[:2])
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        n.forward(x, w, b)
    with pytest.raises(ValueError, match="grad_out: expected"):
        n.backward(x, w, x[:2])
    with pytest.raises(ValueError, match="h_weight: expected"):
        n.double_backward(x, w, x, h_weight=b)
    r = C.Router(8, 2)
    l, ids = torch.zeros(5, 8), torch.zeros(5, 2, dtype=torch.int32)
    with pytest.raises(TypeError, match="logits: expected torch.float32"):
        r.forward(l.bfloat16())
    with pytest.raises(ValueError, match="bias: expected 8"):
        r.forward(l, torch.zeros(7))
    with pytest.raises(TypeError, match="ids: expected torch.int32"):
        r.backward(l, ids.long(), torch.zeros(5, 2))
    with pytest.raises(ValueError, match="grad_weights: expected 10"):
        r.backward(l, ids, torch.zeros(5, 3))
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        r.forward(l)
    dev = torch.device("cuda", 0)
    with pytest.raises(TypeError, match="gates: expected torch.float32"):
        r._gates(torch.zeros(8, 5).double(), "gates", 5, dev)
    with pytest.raises(ValueError, match=r"gates: expected shape \(8, 5\)"):
        r._gates(torch.zeros(5, 8), "gates", 5, dev)
    with pytest.raises(ValueError, match="gates: expected a CUDA tensor"):
        r._gates(torch.zeros(8, 5), "gates", 5, dev)
