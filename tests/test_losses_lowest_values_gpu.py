"""Log-probabilities, and the losses that are taken from them, where logits are finite and as low as their type has them: rows
that a mask of the lowest value has filled, and a chosen token behind such a mask, at temperatures over and under 1.

A softmax sees differences alone, so the bounds are those of the row less its maximum (exact here in 64 bits). What is
chosen far under the maximum has the difference's two roundings, over and under the temperature: logp_error's 6 |logp|
units hold them."""
import math

import numpy as np
import pytest
import torch

import _losses_ref as ref
import zero_gradient_reduction_gb300 as zr
from _losses_ref import BF16, EPS, F16, F32, near

pytestmark = pytest.mark.gpu
INF = float("inf")
LOWEST = {t: torch.finfo(t).min for t in (F32, F16, BF16)}
# a mask's values: a type's lowest, and others that lie far down
FILLS = [(F32, LOWEST[F32]), (F32, -2e30), (F32, -1e31), (F32, -9e29), (BF16, LOWEST[BF16]), (BF16, -2e30), (F16, LOWEST[F16])]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def host(t):
    return t.double().cpu().numpy()


def f32(x):
    return float(np.float32(x))


def scored(z, ids, tau, entropy=None):
    logp = torch.full((z.shape[0],), 7.0, device="cuda")
    zr.token_logprobs(z, ids.cuda(), logp, entropy=entropy, temperature=tau)
    return logp


@pytest.mark.parametrize("V", [1, 2, 9, 300, 50_001])
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_rows_of_nothing_but_a_mask_are_uniform(dtype, fill, V):
    z = torch.full((4, V), fill, dtype=dtype, device="cuda")
    ids = torch.tensor([0, V - 1, V // 2, -1])
    want = np.where(ids.numpy() < 0, 0.0, -math.log(V))
    level = np.zeros((4, V))
    for tau in (1.0, f32(0.7), 1.5, 1e-3, 1e6):
        bound = np.where(ids.numpy() < 0, 0.0, ref.logp_error(level, tau, want))
        entropy = torch.full((4,), 7.0, device="cuda")
        near(scored(z, ids, tau), want, bound, "logp")
        near(scored(z, ids, tau, entropy), want, bound, "logp beside an entropy")
        near(entropy, -want, np.where(ids.numpy() < 0, 0.0, 2 * ref.relative(level, tau) * (2 - want + math.log(V))), "entropy")


@pytest.mark.parametrize("centre,tau,V", [(-2e30, 1.0, 300), (-2e30, 1e6, 50_000), (-1e31, 2.0, 300), (-3e38, f32(0.7), 300)])
def test_rows_far_down_with_differences(centre, tau, V):
    g = torch.Generator().manual_seed(V)
    ulp = float(np.spacing(np.float32(abs(centre))))
    z = (centre + ulp * torch.randint(-6, 7, (6, V), generator=g).double()).float().cuda()
    ids = torch.randint(0, V, (6,), generator=g)
    h = host(z) - host(z).max(1, keepdims=True)
    want = ref.softmax(h, tau)[0][np.arange(6), ids.numpy()]
    for entropy in (None, torch.empty(6, device="cuda")):
        near(scored(z, ids, tau, entropy), want, ref.logp_error(h, tau, want))


@pytest.mark.parametrize("V", [300, 50_000])
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_a_chosen_token_behind_a_mask(dtype, fill, V):
    z, ids = ref.logits(6, V, dtype, torch.Generator().manual_seed(V))
    z[:, V - 10:] = fill
    ids[:3] = V - 4
    ids[3:] = ids[3:].clamp(max=V - 11)
    h = host(z)
    for tau in (1.0, f32(0.7), 1.5, 1e3, 1e-6):
        want = ref.softmax(h, tau)[0][np.arange(6), ids.numpy()]
        bound = ref.logp_error(h, tau, want)
        for entropy in (None, torch.empty(6, device="cuda")):
            got = host(scored(z, ids, tau, entropy))
            beyond = np.abs(want) > torch.finfo(F32).max  # 32 bits have no such number
            assert (got[beyond] == -INF).all() and (np.abs(got - want)[~beyond] <= bound[~beyond]).all(), (tau, got, want)


def test_both_ends_of_the_type():
    """A maximum near the type's largest value over a choice near its lowest: their difference alone has no number."""
    z = torch.full((3, 40), 1e38, device="cuda")
    z[:, 7] = -3e38
    z[1:, 30:] = -INF
    z[2, 7] = -INF
    ids = torch.full((3,), 7)
    for tau in (2.0, 1e3):
        want = -4e38 / tau
        got = host(scored(z, ids, tau))
        assert (np.abs(got[:2] - want) <= 8 * EPS * abs(want)).all() and got[2] == -INF
    assert (host(scored(z, ids, 1.0)) == -INF).all()


@pytest.mark.parametrize("V", [300, 50_001])
@pytest.mark.parametrize("dtype,fill", FILLS)
def test_the_policy_loss_of_masked_rows(dtype, fill, V):
    """The ratio, the KL term and the gradient of rows without a difference."""
    T = 5
    z, ids = torch.full((T, V), fill, dtype=dtype, device="cuda"), torch.tensor([0, V - 1, 17, 8, -1])
    old, near_ref = (torch.full((T,), -math.log(V) + d, device="cuda") for d in (0.05, -0.3))
    adv, weight = torch.tensor([1.0, -0.5, 2.0, -1.5, 1.0], device="cuda"), torch.rand(T, device="cuda") + 0.1
    level = np.zeros((T, V))
    for tau in (1.0, 1.5):
        lo, hi, kl = f32(0.2), f32(0.28), f32(0.1)
        (loss, logp, f), (e_loss, e_logp, e_f) = ref.policy(level, ids.numpy(), host(old), host(adv), host(weight), lo, hi, host(near_ref), kl,
                                                            tau, 1.0)
        got, lp, grad = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(z)
        zr.policy_loss(z, ids.cuda(), old, adv, got, grad, weight=weight, clip=(0.2, 0.28), ref_logp=near_ref, kl=0.1, logp=lp, temperature=tau)
        near(lp, logp, e_logp, "logp")
        near(got, loss, e_loss, "loss")
        at = np.maximum(ids.numpy(), 0)
        near(grad, ref.gradient(level, tau, at, f), ref.gradient_error(level, tau, at, f, e_f, dtype), "gradient")


@pytest.mark.parametrize("dtype,fill", FILLS)
def test_the_policy_loss_of_a_choice_behind_a_mask(dtype, fill):
    """Its ratio is 0: the clipped product counts under an advantage that is negative, and there is no gradient at all."""
    V, tau = 300, 1.5
    z, ids = ref.logits(2, V, dtype, torch.Generator().manual_seed(3))
    z[:, V - 10:] = fill
    ids[:] = V - 4
    want = ref.softmax(host(z), tau)[0][:, V - 4]
    old, adv = torch.full((2,), -6.0, device="cuda"), torch.tensor([1.0, -1.0], device="cuda")
    loss, lp, grad = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.full_like(z, 7.0)
    zr.policy_loss(z, ids.cuda(), old, adv, loss, grad, clip=(0.2, 0.28), logp=lp, temperature=tau)
    near(lp, want, ref.logp_error(host(z), tau, want))
    assert float(loss[0]) == 0 and abs(float(loss[1]) - 0.8) <= 8 * EPS and bool((grad == 0).all())


@pytest.mark.parametrize("dtype,fill", FILLS)
def test_the_preference_loss_of_masked_rows(dtype, fill):
    """One row of each sequence filled with the mask: rewards, loss and gradients as of rows of zeros."""
    V, lengths, beta, smoothing = 300, (3, 2, 4, 1), 0.3, 0.1
    g = torch.Generator().manual_seed(4)
    T, starts = sum(lengths), np.concatenate([[0], np.cumsum(lengths)])
    z, ids = ref.logits(T, V, dtype, g)
    level = z.clone()
    z[starts[:-1].tolist()], level[starts[:-1].tolist()] = fill, 0.0
    h, w = host(level), np.ones(2)
    near_ref = torch.from_numpy(ref.softmax(h, 1.0)[0][np.arange(T), ids.numpy()] + 0.5 * torch.randn(T, generator=g).double().numpy()).float().cuda()
    for tau in (1.0, 1.5):
        (loss, rewards, f, _), (e_loss, e_rewards, e_f) = ref.preference(h, ids.numpy(), starts, host(near_ref), w, f32(beta), f32(smoothing), tau, 1.0)
        got, r, grad = torch.empty(2, device="cuda"), torch.empty(4, device="cuda"), torch.empty_like(z)
        work = torch.empty(zr.preference_bytes(T, 2), dtype=torch.uint8, device="cuda")
        zr.preference_loss(z, ids.cuda(), torch.from_numpy(starts).cuda(), near_ref, got, work, grad, beta=beta, smoothing=smoothing, rewards=r,
                           temperature=tau)
        near(r, rewards, e_rewards, "rewards")
        near(got, loss, e_loss, "loss")
        near(grad, ref.gradient(h, tau, ids.numpy(), f), ref.gradient_error(h, tau, ids.numpy(), f, e_f, dtype), "gradient")


@pytest.mark.parametrize("dtype,fill", FILLS)
def test_the_reward_of_a_choice_behind_a_mask(dtype, fill):
    """A choice far down decides its sequence's reward and the pair's margin, by beta / tau of it."""
    V, beta, tau = 300, 0.1, 1.5
    z, ids = ref.logits(4, V, dtype, torch.Generator().manual_seed(5))
    z[:, V - 10:] = fill
    ids = ids.clamp(max=V - 11)
    ids[0] = V - 4
    starts, near_ref = np.array([0, 2, 4]), torch.zeros(4, device="cuda")
    with np.errstate(all="ignore"):  # the slope's error at a margin of 10^30, which is not looked at
        (loss, rewards, _, _), (e_loss, e_rewards, _) = ref.preference(host(z), ids.numpy(), starts, np.zeros(4), np.ones(1), f32(beta), 0.0, tau, 1.0)
    got, r = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    work = torch.empty(zr.preference_bytes(4, 1), dtype=torch.uint8, device="cuda")
    zr.preference_loss(z, ids.cuda(), torch.from_numpy(starts).cuda(), near_ref, got, work, beta=beta, rewards=r, temperature=tau)
    near(r, rewards, e_rewards, "rewards")
    near(got, loss, e_loss, "loss")
