"""The chosen tokens' log-probabilities, and the clipped policy loss with its gradient, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import _losses_ref as ref
import zero_gradient_reduction_gb300 as zr
from _losses_ref import BF16, F16, F32, near

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ log-probabilities
def check_logprobs(z, ids, tau, ids_type=torch.int64):
    T = z.shape[0]
    logp, entropy = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    zr.token_logprobs(z, ids.to(ids_type).cuda(), logp, entropy=entropy, temperature=tau)
    alone = torch.full((T,), 7.0, device="cuda")
    zr.token_logprobs(z, ids.to(ids_type).cuda(), alone, temperature=tau)
    h, a = host(z), ids.numpy()
    logq, q = ref.softmax(h, tau)
    want = np.where(a < 0, 0.0, logq[np.arange(T), np.maximum(a, 0)])
    bound = np.where(a < 0, 0.0, ref.logp_error(h, tau, want))
    near(logp, want, bound, "logp")
    near(alone, want, bound, "logp without an entropy")
    with np.errstate(invalid="ignore"):
        H = np.where(a < 0, 0.0, -np.where(q > 0, q * logq, 0.0).sum(1))
    # log S less the mean exponent: E of the sum, E and 3 A roundings of the terms times their exponents
    near(entropy, H, np.where(a < 0, 0.0, 2 * ref.relative(h, tau) * (2 + H + math.log(z.shape[1]))), "entropy")


@pytest.mark.parametrize("T,V", [(1, 1), (1, 7), (5, 8), (9, 33), (7, 1000), (3, 5001), (40, 4096), (2, 50257), (400, 2000), (1, 300_001)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_logprobs(T, V, dtype):
    z, ids = ref.logits(T, V, dtype, torch.Generator().manual_seed(T + V))
    if T > 3:
        ids[1] = -1
    for tau, kind in ((1.0, torch.int64), (0.6, torch.int32)):
        check_logprobs(z, ids, tau, kind)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld", [1001, 1003, 1008])
def test_logprobs_row_strides(dtype, ld):
    z, ids = ref.logits(12, 1001, dtype, torch.Generator().manual_seed(ld), ld=ld)
    check_logprobs(z, ids, 1.0)


@pytest.mark.parametrize("at", [0, 1, 7, 8, 9, 500, 1000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_logprobs_of_each_place_in_a_row(dtype, at):
    """The chosen column among the values before, in and behind the whole words of rows that begin anywhere."""
    z, ids = ref.logits(9, 1001, dtype, torch.Generator().manual_seed(at), ld=1003)
    check_logprobs(z, torch.full_like(ids, at), 1.0)


def test_logprobs_of_almost_certain_tokens():
    """1 - q down to 10^-30: the logarithm keeps E of itself, which log(1 - small) from the whole sum could not."""
    V, T = 1000, 12
    z = torch.zeros(T, V)
    z[:, 17] = torch.linspace(8, 75, T)
    logp = torch.empty(T, device="cuda")
    zr.token_logprobs(z.cuda(), torch.full((T,), 17, device="cuda"), logp)
    want = -np.log1p((V - 1) * np.exp(-z[:, 17].double().numpy()))
    assert (np.abs(host(logp) - want) <= np.abs(want) * (2 * ref.relative(host(z), 1.0) + 8 * ref.EPS)).all()


def test_errors_of_many_tokens_have_no_common_sign():
    """A sequence's sum of log-probabilities: the mean error of 4000 tokens lies under a tenth of what each may have."""
    T, V = 4000, 3000
    z, ids = ref.logits(T, V, BF16, torch.Generator().manual_seed(3), certain=1.0)
    for tau in (1.0, float(np.float32(0.7))):  # as the call takes it
        logp = torch.empty(T, device="cuda")
        zr.token_logprobs(z, ids.cuda(), logp, temperature=tau)
        h = host(z)
        d = host(logp) - ref.softmax(h, tau)[0][np.arange(T), ids.numpy()]
        # a logp of up to 16 is rounded to 2^-21 (an rms of 1.4e-7), with a few roundings of the like before it; their mean
        # has an rms 63 times smaller, and what they all share may be as much again
        assert abs(d.mean()) < 4e-8 and np.sqrt((d ** 2).mean()) < 1e-6


def test_logprobs_masks_and_rows_without_an_answer():
    for V in (130, 50_000):
        z, ids = ref.logits(9, V, F32, torch.Generator().manual_seed(V))
        ids = ids.clamp(max=V // 2)
        z[:, V - 20:] = -INF
        z[:, V - 40:V - 20] = torch.finfo(F32).min
        check_logprobs(z, ids, 1.0)
        chosen = ids.clone()
        chosen[0] = V - 1                                       # chosen, but masked
        z[1, V - 1], z[2, 3], z[3] = NAN, INF, -INF             # no number, infinite, all masked
        chosen[4] = V                                           # past the vocabulary
        chosen[5] = (1 << 32) + 5
        z[6], chosen[6] = NAN, -1                               # not scored, whatever it holds
        logp, entropy = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        zr.token_logprobs(z, chosen.cuda(), logp, entropy=entropy)
        assert float(logp[0]) == -INF and float(entropy[0]) > 0
        assert torch.isnan(logp).tolist() == [False, True, True, True, True, True, False, False, False]
        assert torch.isnan(entropy).tolist() == [False, True, True, True, True, True, False, False, False]
        assert float(logp[6]) == 0 and float(entropy[6]) == 0


def test_logprobs_masked_at_temperatures_of_every_scale():
    """log2(e)/tau whose upper bits alone are above it, at or under it: masked logits have no part in any of them."""
    c = 1.4426950408889634
    near_12_bits = [np.float32(c / k) for k in (np.arange(2048, 2300) / 2048)]
    tau = [t for base in near_12_bits for t in (np.nextafter(base, np.float32(0)), base, np.nextafter(base, np.float32(9)))]
    above = [t for t in tau if np.float32(c / t).view(np.uint32) & 0xFFF == 0 and float(np.float32(c / t)) > c / float(t)]
    assert above
    z, ids = ref.logits(8, 700, BF16, torch.Generator().manual_seed(2))
    ids = ids.clamp(max=300)
    z[:, 400:] = -INF
    for t in above[:8] + tau[:8] + [1e-6, 1e6]:
        check_logprobs(z if t > 1e-3 else (z * 1e-6).to(F32), ids, float(np.float32(t)))


@pytest.mark.parametrize("centre,tau,V", [(5000.0, 0.01, 900), (6931.0, 0.01, 60_000), (-3e4, 1e-3, 500), (1e30, 1.0, 300)])
def test_logprobs_far_from_zero_at_low_temperatures(centre, tau, V):
    """Exponents whose common part is from 10^5 to 10^30: the spread decides what fp32 may cost."""
    g = torch.Generator().manual_seed(V)
    ulp = float(np.spacing(np.float32(abs(centre))))
    z = (centre + max(ulp, tau) * torch.randint(-6, 7, (6, V), generator=g).double()).float().cuda()
    ids = torch.randint(0, V, (6,), generator=g)
    logp, entropy = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    zr.token_logprobs(z, ids.cuda(), logp, entropy=entropy, temperature=tau)
    h = host(z) - host(z).max(1, keepdims=True)
    logq, q = ref.softmax(h, tau)
    want = logq[np.arange(6), ids.numpy()]
    near(logp, want, ref.logp_error(h, tau, want))
    H = -np.where(q > 0, q * logq, 0.0).sum(1)
    near(entropy, H, 2 * ref.relative(h, tau) * (2 + H + math.log(V)))


# ------------------------------------------------------------------ the policy loss
def case(T, V, dtype, seed, tau=1.0, lo=0.2, hi=0.28, ld=None):
    g = torch.Generator().manual_seed(seed)
    z, ids = ref.logits(T, V, dtype, g, ld=ld)
    h = host(z)
    logp = ref.softmax(h, tau)[0][np.arange(T), ids.numpy()]
    step = 0.3 * torch.randn(T, generator=g).double().numpy()
    for border in (math.log(1 - lo), math.log1p(hi)):  # the gradient jumps there
        step = np.where(np.abs(step - border) < 1e-2, border + 2e-2, step)
    old = torch.from_numpy(logp - step).float()
    near_ref = torch.from_numpy(logp + 0.3 * torch.randn(T, generator=g).double().numpy()).float()
    adv, weight = torch.randn(T, generator=g), torch.rand(T, generator=g) + 0.1
    if T > 3:
        weight[1], ids[2], adv[3] = 0, -1, 0
    return z, ids, old.cuda(), adv.cuda(), weight.cuda(), near_ref.cuda()


def check(z, ids, old, adv, weight, near_ref, tau=1.0, scale=1.0, lo=0.2, hi=0.28, kl=0.1, grad=None, in_place=False, plan=None, S=1.0):
    T = z.shape[0]
    h = host(z)
    (loss, logp, f), (e_loss, e_logp, e_f) = ref.policy(h, ids.numpy(), host(old), host(adv), host(weight), float(np.float32(lo)),
                                                         float(np.float32(hi)), host(near_ref), float(np.float32(kl)), tau, scale * S)
    out = z if in_place else torch.full_like(z, 7.0) if grad is None else grad
    got, lp = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    zr.policy_loss(z, ids.cuda(), old, adv, got, out, weight=weight, clip=(lo, hi), ref_logp=near_ref if kl else None, kl=kl, logp=lp,
                   temperature=tau, grad_scale=scale, plan=plan)
    near(got, loss, e_loss, "loss")
    near(lp, logp, e_logp, "logp")
    at = np.maximum(ids.numpy(), 0)
    near(out, ref.gradient(h, tau, at, f), ref.gradient_error(h, tau, at, f, e_f, z.dtype), "gradient")
    return got, out


@pytest.mark.parametrize("T,V", [(1, 1), (1, 7), (5, 8), (9, 33), (7, 1000), (3, 5001), (40, 4096), (2, 50257)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_loss_and_gradient(T, V, dtype):
    for i, (tau, kl) in enumerate(((1.0, 0.0), (0.7, 0.1), (1.5, 0.5))):
        check(*case(T, V, dtype, seed=T + V + i, tau=tau), tau=tau, kl=kl, scale=3.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_and_long_rows(dtype):
    check(*case(400, 2000, dtype, seed=1))       # a block for each row, several waves
    check(*case(1, 300_000, dtype, seed=2))      # a row for a cluster
    check(*case(1, 600_001, dtype, seed=3))      # more than a cluster's shared memory in 32 bits


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ldz,ldg", [(1003, 1003), (1003, 1001), (1008, 1003), (1001, 1008)])
def test_row_strides(dtype, ldz, ldg):
    room = torch.full((12, ldg), 7.0, dtype=dtype, device="cuda")
    check(*case(12, 1001, dtype, seed=ldz, ld=ldz), grad=room[:, :1001])
    assert bool((room[:, 1001:] == 7.0).all())


@pytest.mark.parametrize("at", [0, 1, 7, 8, 9, 500, 1000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_each_place_in_a_row(dtype, at):
    z, ids, *rest = case(9, 1001, dtype, seed=at, ld=1003)
    check(z, torch.where(ids < 0, ids, at), *rest, kl=0.0)


@pytest.mark.parametrize("V", [1000, 1001, 60_000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_gradient_over_the_logits(V, dtype):
    check(*case(6, V, dtype, seed=V), in_place=True, scale=2.0)


def test_gradient_over_the_logits_longer_than_shared_memory():
    check(*case(1, 600_001, F32, seed=3), in_place=True)


def test_both_sides_of_the_clip():
    """Ratios far under, in and far over the range, under advantages of both signs; one-sided ranges and none."""
    T, V = 40, 300
    z, ids, _, _, weight, near_ref = case(T, V, F32, seed=4)
    ids = ids.clamp(min=0)
    weight[:] = 1
    logp = ref.softmax(host(z), 1.0)[0][np.arange(T), ids.numpy()]
    adv = torch.where(torch.arange(T) % 2 == 0, 1.5, -0.5).cuda()
    old = torch.from_numpy(logp - np.linspace(-3, 3, T)).float().cuda()
    for lo, hi in ((0.2, 0.28), (0.0, 0.5), (1.0, 3.0), (1.0, 1e30)):
        ratio = np.exp(logp - host(old))
        assert (np.abs(ratio - (1 - lo)) > 1e-3).all() and (np.abs(ratio - (1 + hi)) > 1e-3).all()
        check(z, ids, old, adv, weight, near_ref, lo=lo, hi=hi, kl=0.0)
    loss, grad = torch.empty(T, device="cuda"), torch.empty_like(z)
    zr.policy_loss(z, ids.cuda(), old, adv, loss, grad, clip=(0.2, 0.2))
    assert bool((grad[-2] == 0).all()) and bool((grad[1] == 0).all())  # clipped: no gradient at all
    assert bool((grad[0] != 0).any()) and bool((grad[-1] != 0).any())


def test_almost_certain_tokens_keep_their_gradient():
    """1 - q down to 10^-30 in fp32, with its own relative accuracy."""
    T, V = 12, 500
    z = torch.zeros(T, V)
    z[:, 3] = torch.linspace(8, 75, T)
    ids = torch.full((T,), 3)
    h = z.double().numpy()
    logp = ref.softmax(h, 1.0)[0][:, 3]
    old = torch.from_numpy(logp).float().cuda()
    loss, grad = torch.empty(T, device="cuda"), torch.empty(T, V, device="cuda")
    zr.policy_loss(z.cuda(), ids.cuda(), old, torch.ones(T, device="cuda"), loss, grad)
    want = -ref.others(h, 1.0, ids.numpy())
    rel = 2 * ref.relative(h, 1.0) + ref.logp_error(h, 1.0, logp) + 16 * ref.EPS
    assert (np.abs(host(grad[:, 3]) - want) <= np.abs(want) * rel).all()


def test_masked_vocabulary():
    for V in (300, 50_000):
        z, ids, *rest = case(8, V, BF16, seed=5)
        ids = ids.clamp(max=V // 2)
        z[:, V - 50:] = -INF
        z[:, V - 100:V - 50] = torch.finfo(BF16).min
        _, grad = check(z, ids, *rest, kl=0.0)
        assert bool((grad[:, V - 100:] == 0).all())


def test_rows_without_loss_are_not_read():
    z, ids, old, adv, weight, near_ref = case(6, 130, F32, seed=6)
    weight[:] = 1
    weight[0], ids[1] = 0, -1
    z[0], z[1] = NAN, INF
    old[0], adv[1] = NAN, NAN
    ids[2] = 5
    loss, logp, grad = torch.full((6,), 7.0, device="cuda"), torch.full((6,), 7.0, device="cuda"), torch.full_like(z, 7.0)
    zr.policy_loss(z, ids.cuda(), old, adv, loss, grad, weight=weight, logp=logp)
    for out in (loss, logp, grad):
        assert bool((out[:2] == 0).all()) and bool(torch.isfinite(out).all())


def test_rows_that_have_no_answer_say_so():
    for V in (130, 50_000):
        z, ids, old, adv, weight, near_ref = case(10, V, F32, seed=7)
        weight[:], adv[:] = 1, 1
        ids = ids.clamp(min=0)
        z[0, V - 1], z[1, 3], z[2] = NAN, INF, -INF
        ids[3] = V
        old[4], adv[5], weight[6] = NAN, NAN, NAN
        near_ref[7] = NAN
        loss, grad = torch.empty(10, device="cuda"), torch.empty_like(z)
        zr.policy_loss(z, ids.cuda(), old, adv, loss, grad, weight=weight, ref_logp=near_ref, kl=0.1)
        assert torch.isnan(loss).tolist() == [True] * 8 + [False] * 2
        assert torch.isnan(grad).all(1).tolist() == [True] * 8 + [False] * 2
        assert bool(torch.isfinite(grad[8:]).all())


def test_a_reference_without_a_kl_term_is_not_read():
    z, ids, old, adv, weight, near_ref = case(5, 64, F32, seed=8)
    near_ref[:] = NAN
    loss = torch.empty(5, device="cuda")
    zr.policy_loss(z, ids.cuda(), old, adv, loss, weight=weight, ref_logp=near_ref, kl=0.0)
    assert bool(torch.isfinite(loss).all())


def test_gradient_against_differences():
    """The loss's own differences in 64 bits, at logits moved both ways: the formula of the gradient, not its rounding."""
    T, V, h = 4, 9, 1e-5
    z, ids, old, adv, weight, near_ref = case(T, V, F32, seed=9, tau=0.8)
    weight[:], adv[:] = torch.rand(T).cuda() + 0.5, torch.tensor([1.0, -1.0, 0.5, -2.0]).cuda()
    ids = ids.clamp(min=0)
    loss, grad = torch.empty(T, device="cuda"), torch.empty_like(z)
    zr.policy_loss(z, ids.cuda(), old, adv, loss, grad, weight=weight, ref_logp=near_ref, kl=0.3, temperature=0.8)

    def total(x):
        return ref.policy(x, ids.numpy(), host(old), host(adv), host(weight), float(np.float32(0.2)), float(np.float32(0.2)), host(near_ref),
                          float(np.float32(0.3)), 0.8, 1.0)[0][0]

    x = host(z)
    for v in range(V):
        up, down = x.copy(), x.copy()
        up[:, v] += h
        down[:, v] -= h
        slope = (total(up) - total(down)) / (2 * h)
        assert (np.abs(host(grad[:, v]) - slope) <= 1e-4 * np.abs(host(grad)).max(1) + 1e-7).all()


def test_the_plans_loss_scale():
    plan = zr.Plan([64], W=1, dtype=zr.F16, stage=1, cap=64, scaler=zr.Scaler(init_scale=512.0))
    check(*case(5, 100, F32, seed=10), plan=plan, scale=2.0, S=512.0)
    plan.close()


def test_offsets_past_32_bits():
    T, V = 44_000, 50_304
    z = torch.empty(T, V, dtype=BF16, device="cuda").normal_()
    assert z.numel() > 1 << 31
    some = torch.tensor([0, 21_000, T - 2, T - 1])
    ids = torch.randint(0, V, (T,), device="cuda")
    h, a = host(z[some.cuda()]), ids[some.cuda()].cpu()
    logp = ref.softmax(h, 1.0)[0][np.arange(4), a.numpy()]
    old = torch.full((T,), -11.0, device="cuda")
    old[some.cuda()] = torch.from_numpy(logp - 0.1).float().cuda()
    adv, ones = torch.ones(T, device="cuda"), torch.ones(T, device="cuda")
    lp = torch.empty(T, device="cuda")
    zr.token_logprobs(z, ids, lp)
    near(lp[some.cuda()], logp, ref.logp_error(h, 1.0, logp))
    loss = torch.empty(T, device="cuda")
    zr.policy_loss(z, ids, old, adv, loss, z, weight=ones, grad_scale=64.0)
    pick = [host(v[some.cuda()]) for v in (old, adv, ones)]
    clip = float(np.float32(0.2))
    (want, _, f), (e, _, e_f) = ref.policy(h, a.numpy(), *pick, clip, clip, np.zeros(4), 0.0, 1.0, 64.0)
    near(loss[some.cuda()], want, e)
    near(z[some.cuda()], ref.gradient(h, 1.0, a.numpy(), f), ref.gradient_error(h, 1.0, a.numpy(), f, e_f, BF16))


def test_captured_and_on_another_stream():
    """A captured pass replayed on new logits, and a pass on a side stream, give the bytes of a plain call."""
    z, ids, old, adv, weight, near_ref = case(30, 3000, BF16, seed=11)
    ids = ids.cuda()
    outs = [torch.empty(30, device="cuda"), torch.empty(30, device="cuda"), torch.empty_like(z), torch.empty(30, device="cuda")]

    def call(o, stream=None):
        zr.token_logprobs(z, ids, o[0], entropy=o[3], stream=stream)
        zr.policy_loss(z, ids, old, adv, o[1], o[2], weight=weight, ref_logp=near_ref, kl=0.1, stream=stream)

    call(outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    z.copy_(z.flip(0))
    plain = [torch.empty_like(o) for o in outs]
    call(plain)
    for o in outs:
        o.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    side = torch.cuda.Stream()
    other = [torch.full_like(o, 7.0) for o in outs]
    side.wait_stream(torch.cuda.current_stream())
    call(other, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, plain))


def test_no_rows():
    z, empty = torch.empty(0, 50, device="cuda"), torch.empty(0, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    zr.token_logprobs(z, ids, empty)
    zr.policy_loss(z, ids, empty, empty, empty, z)
