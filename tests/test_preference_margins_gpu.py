"""The preference loss over its margin: far out on both sides, infinite, and of a pair that does not count.

Against the definition -(1 - l) log S(m) - l log S(-m) in 64 bits, at the margin of the rewards that the call returns. Both
terms are at or over 0, so nothing cancels: an exponential (2 units of 2^-23), a logarithm (1), the coefficient, a product, a
sum and the weight (5 halves) are under 16 times 2^-24 of the loss itself."""
import numpy as np
import pytest
import torch

import _losses_ref as ref
import zero_gradient_reduction_gb300 as zr
from _losses_ref import EPS, F32

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def run(z, ids, starts, near_ref, weight=None, **kw):
    pairs = (len(starts) - 1) // 2
    loss, r, grad = torch.full((pairs,), 7.0, device="cuda"), torch.full((2 * pairs,), 7.0, device="cuda"), torch.full_like(z, 7.0)
    work = torch.empty(zr.preference_bytes(z.shape[0], pairs), dtype=torch.uint8, device="cuda")
    zr.preference_loss(z, ids.cuda(), torch.tensor(starts, device="cuda"), near_ref, loss, work, grad, weight=weight, rewards=r, **kw)
    return loss, r, grad


@pytest.mark.parametrize("smoothing", [0.0, 1e-3, 0.1, 0.5, 0.9, 1.0])
def test_margins_of_every_size(smoothing):
    m = np.array([-300, -80, -30, -17, -9, -3, -1, -0.3, -1e-3, 0, 1e-3, 0.3, 1, 3, 9, 17, 30, 80, 300], np.float64)
    T = 2 * len(m)
    z, ids = ref.logits(T, 20, F32, torch.Generator().manual_seed(1))
    logp = ref.softmax(z.double().cpu().numpy(), 1.0)[0][np.arange(T), ids.numpy()]
    near_ref = torch.from_numpy(logp - np.stack([m / 2, -m / 2], 1).reshape(-1)).float().cuda()
    loss, r, grad = run(z, ids, list(range(T + 1)), near_ref, beta=1.0, smoothing=smoothing)
    r = r.cpu().numpy()
    margin = (r[0::2] - r[1::2]).astype(np.float64)  # rounded to 32 bits, as the margin is
    assert (np.abs(margin - m) < 1e-4).all()
    lam = float(np.float32(smoothing))
    want = (1 - lam) * np.logaddexp(0, -margin) + lam * np.logaddexp(0, margin)
    got = loss.double().cpu().numpy()
    assert (np.abs(got - want) <= 16 * EPS * want + 2.0 ** -126).all(), (got, want)
    assert bool(torch.isfinite(grad).all())


@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
def test_a_masked_token_on_either_side(smoothing):
    """An infinite margin: the side that is wrong has an infinite loss where it counts at all, and gradients are finite."""
    z, ids = ref.logits(8, 50, F32, torch.Generator().manual_seed(2))
    ids = ids.clamp(max=40)
    ids[1] = ids[6] = 45  # in the preferred sequence of the first pair, in the other of the second
    z[:, 45] = -INF
    loss, r, grad = run(z, ids, [0, 2, 4, 6, 8], torch.zeros(8, device="cuda"), smoothing=smoothing)
    assert r[0] == -INF and r[3] == -INF and bool(torch.isfinite(r[1:3]).all())
    assert loss.tolist() == [INF if smoothing < 1 else 0.0, INF if smoothing > 0 else 0.0]
    assert bool(torch.isfinite(grad).all())


def test_a_margin_that_is_no_number_stays_so():
    z, ids = ref.logits(4, 50, F32, torch.Generator().manual_seed(3))
    for smoothing in (0.0, 0.3, 1.0):
        near_ref = torch.zeros(4, device="cuda")
        near_ref[0] = NAN
        loss, _, _ = run(z, ids, [0, 1, 2, 3, 4], near_ref, smoothing=smoothing)
        assert torch.isnan(loss).tolist() == [True, False]


def test_a_pair_that_does_not_count_says_nothing_of_its_starts():
    """Weight 0 goes before starts that do not ascend, for the loss and the rewards alike; the other pairs are as they were."""
    z, ids = ref.logits(9, 30, F32, torch.Generator().manual_seed(4))
    near_ref = torch.zeros(9, device="cuda")
    for bad in ([5, 3, 5], [-1, 0, 5], [0, 40, 5]):
        for weight in ([0.0, 1.0], [1.0, 1.0], [0.0, 0.0]):
            loss, r, _ = run(z, ids, [*bad, 7, 9], near_ref, weight=torch.tensor(weight, device="cuda"))
            want = 0.0 if weight[0] == 0 else NAN
            assert all(np.array_equal(float(v), want, equal_nan=True) for v in (loss[0], r[0], r[1])), (bad, weight, loss, r)
            assert bool(torch.isfinite(loss[1])) and bool(torch.isfinite(r[2:]).all()) and (float(loss[1]) > 0) == (weight[1] > 0)
