"""Calls of the layer norm and the router on a stream that is not the current
one, while the current stream works with memory of its own.

Everything that such a call allocates (its workspace, its new outputs) is used
by the stream it is given, so it must not be memory that the current stream
still reads or has been given again.  One of the two streams is held back by
a kernel that only waits, so that the order is that of the test.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HOLD = 20_000_000  # clock ticks, some 10 ms


def C():
    from equivariant_mlip_clebsch_b200 import cgtp
    return cgtp


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def test_workspace_is_the_calls_own_until_it_has_run(dev):
    """Memory that the current stream is given after the call keeps what it writes."""
    norm = C().LayerNorm("256x0e")
    n = 20_000
    x, g = torch.randn(n, norm.d, device=dev), torch.randn(n, norm.d, device=dev)
    ref = norm.backward(x, None, g), norm.double_backward(x, None, g, g)
    size = norm.workspace_size(n)
    assert size > 0
    side = torch.cuda.Stream()
    for call, want in ((norm.backward, ref[0]), (lambda *a, **k: norm.double_backward(*a, g, **k), ref[1])):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD)
        out = call(x, None, g, stream=side)
        mine = [torch.full((size,), 7, dtype=torch.uint8, device=dev) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in mine)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_new_outputs_are_not_memory_that_the_current_stream_reads(dev):
    """Arrays dropped while the current stream has yet to read them."""
    n = 20_000
    norm, router = C().LayerNorm("64x0e"), C().Router(64, 4)
    x, g = torch.randn(n, 64, device=dev), torch.randn(n, 64, device=dev)
    ids = router.forward(x)[0]
    side = torch.cuda.Stream()
    calls = (lambda: norm.forward(x, stream=side), lambda: norm.backward(x, None, g, stream=side),
             lambda: norm.double_backward(x, None, g, g, stream=side), lambda: router.forward(x, stream=side),
             lambda: router.backward(x, ids, grad_gates=g.view(64, n), stream=side))
    for call in calls:
        call()
        torch.cuda.synchronize()
        read = torch.zeros(4, device=dev)
        dropped = [torch.full((n, 64), 3.0, device=dev) for _ in range(4)]
        torch.cuda.synchronize()
        torch.cuda._sleep(HOLD)
        for i, t in enumerate(dropped):
            torch.amax((t - 3.0).abs(), dim=(0, 1), out=read[i])
        del dropped, t
        out = call()
        torch.cuda.synchronize()
        assert read.tolist() == [0.0] * 4
        del out
