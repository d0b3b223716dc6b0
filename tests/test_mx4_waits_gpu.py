"""The products' bounded waits: when their clocks run, and who hears of one that ran out."""
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr
from test_mx4_gpu import check, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    zr.mx4_status()


def stalled(call):
    """One call whose waits run out after two seconds each."""
    zr.lib().zr_mx4_stall_waits(1)
    try:
        call()
    finally:
        zr.lib().zr_mx4_stall_waits(0)


@pytest.mark.parametrize("M,N,K", [(100, 300, 700), (64, 512, 8192), (1024, 4096, 4096)])
def test_the_launch_before_does_not_use_up_a_products_time(M, N, K):
    """A product by blocks alone, by clusters that share K, and by pairs begins while the one before it still runs, for
    the four seconds that its waits and the waits for its copies take: it waits that long and is right."""
    (a, _), (b, _) = quantised(64, 200, 1), quantised(64, 200, 2)
    (c, cv), (d, dv) = quantised(M, K, 3), quantised(N, K, 4)
    first, out = torch.empty(64, 64, device="cuda"), torch.full((M, N), 7.0, device="cuda")
    zr.mx4_matmul(c, d, out)  # loaded before
    out.fill_(7.0)
    torch.cuda.synchronize()
    stalled(lambda: zr.mx4_matmul(a, b, first))
    zr.mx4_matmul(c, d, out)
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5  # the first one's
    zr.mx4_status()
    check(out[:, :400], cv, dv[:400])


def test_every_stream_hears_of_a_wait_that_ran_out():
    """A report that one stream has had is not lost to another: the product's own, above all."""
    (a, _), (b, _) = quantised(64, 200, 1), quantised(64, 200, 2)
    out, side, other = torch.empty(64, 64, device="cuda"), torch.cuda.Stream(), torch.cuda.Stream()
    for s in (None, side, other):
        try:
            zr.mx4_status(stream=s)
        except zr.ZrError:
            pass  # of another test, if at all
    torch.cuda.synchronize()
    stalled(lambda: zr.mx4_matmul(a, b, out, stream=side))
    side.synchronize()
    for s in (None, other, side):
        with pytest.raises(zr.ZrError) as e:
            zr.mx4_status(stream=s)
        assert e.value.status == 5
    for s in (side, None, other):
        zr.mx4_status(stream=s)


def test_a_replayed_product_is_heard_of_where_it_ran():
    """Captured on one stream, replayed on another: the stream of the replay hears of it."""
    (a, _), (b, _) = quantised(64, 200, 1), quantised(64, 200, 2)
    out, side, graph = torch.empty(64, 64, device="cuda"), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    zr.mx4_matmul(a, b, out)
    torch.cuda.synchronize()

    def capture():
        with torch.cuda.graph(graph, stream=side):
            zr.mx4_matmul(a, b, out, stream=side)

    stalled(capture)
    zr.mx4_status()
    graph.replay()
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5
    zr.mx4_status()
