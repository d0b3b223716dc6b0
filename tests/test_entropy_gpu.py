"""The entropy of rows with hardly any: rows that are almost certain."""
import math

import numpy as np
import pytest
import torch

import _losses_ref as ref
import zero_gradient_reduction_gb300 as zr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def rows(V, column, tau=1.0):
    """Zeros but for one column, which is chosen by odds of e^8 to e^75 to one of the others; and their entropy:
    with P = (V - 1) e^-z, log(1 + P) + z P / (1 + P)."""
    z = torch.zeros(200, V)
    z[:, column] = torch.linspace(8, 75, 200) * tau
    x = z[:, column].double().numpy() / tau
    odds = (V - 1) * np.exp(-x)
    return z, np.log1p(odds) + x * odds / (1 + odds)


def entropies(z, ids, tau=1.0):
    T = z.shape[0]
    logp, entropy = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    zr.token_logprobs(z.cuda(), ids.cuda(), logp, entropy=entropy, temperature=tau)
    return entropy.double().cpu().numpy()


@pytest.mark.parametrize("V,column,tau", [(1000, 17, 1.0), (1000, 999, 0.5), (50_000, 30_000, 1.0)])
def test_almost_certain_choices_keep_their_entropy(V, column, tau):
    """Down to 10^-27: as the log-probability, an almost certain choice's entropy keeps its relative accuracy. E for the
    sum of the others, E for that of their distances to the choice, whose own 3 roundings of 1.45 z are under another, and
    ten units for what joins them."""
    z, want = rows(V, column, tau)
    got = entropies(z, torch.full((200,), column), tau)
    assert (np.abs(got - want) <= want * (3 * ref.relative(z.double().numpy(), tau) + 10 * ref.EPS)).all()


@pytest.mark.parametrize("V", [2, 1000, 50_000])
def test_no_entropy_is_under_zero(V):
    """Where another token than the chosen one has almost everything, the entropy is right to some 2^-24 of 1, and not
    negative; where a row has one token alone it is 0."""
    z, want = rows(V, 1)
    got = entropies(z, torch.zeros(200, dtype=torch.int64))
    assert (got >= 0).all()
    assert (np.abs(got - want) <= 2 * ref.relative(z.double().numpy(), 1.0) * (2 + want + math.log(V))).all()
    z[:, 2:], z[:, 0] = -float("inf"), -float("inf")
    for chosen in (0, 1):
        got = entropies(z, torch.full((200,), chosen))
        assert (got >= 0).all() and (got <= 2.0 ** -21).all()
    assert (got == 0).all()
