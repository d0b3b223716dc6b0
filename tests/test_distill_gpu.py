"""The distillation loss against a teacher's top logits, and its gradient, against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def formula(z, ids, teacher, weight, tau, scale):
    """(loss [T], grad [T, V], p [T, V]: what the teacher puts on each column) in 64 bits, row by row."""
    T, V = z.shape
    loss, grad, onto = np.zeros(T), np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        kept = (ids[t] >= 0) & ~np.isneginf(teacher[t])
        if weight[t] == 0 or not kept.any():
            continue
        a = teacher[t][kept] / tau
        lp = a - a.max() - np.log(np.exp(a - a.max()).sum())
        with np.errstate(invalid="ignore"):
            b = z[t] / tau
            lq = b - b.max() - np.log(np.exp(b - b.max()).sum())
        p = np.exp(lp)
        np.add.at(onto[t], ids[t][kept], p)
        loss[t] = weight[t] * tau ** 2 * (p * (lp - lq[ids[t][kept]])).sum()
        grad[t] = weight[t] * tau * scale * (np.exp(lq) - onto[t])
    return loss, grad, onto


def bounds(z, teacher, loss, grad, onto, weight, tau, scale, dtype):
    """What fp32 may cost. An exponent z/tau log2(e) - max carries three roundings of terms up to A = max |z| log2(e)/tau,
    2^2 units of exp2 and the sum's roundings (each thread's terms in eight, then threads: under 100 additions); the
    gradient's q and p each have that relative error, then one rounding to the type. The loss adds the logarithms'."""
    A = (np.abs(np.where(np.isfinite(z), z, 0)).max() + np.abs(np.where(np.isfinite(teacher), teacher, 0)).max()) * 1.45 / tau
    eps = 2.0 ** -24 * (6 * A + 150)
    f = np.abs(weight * tau * scale)[:, None]
    g = eps * (np.abs(grad) + 2 * f * onto)
    # the loss is a mean under p of differences of logarithms, each an exponent less a logarithm
    l = np.abs(weight) * tau ** 2 * (2 * eps * (A + 20)) + eps * np.abs(loss)
    return l, g + ref.rounding(dtype, np.abs(grad) + g) * (1 + 2.0 ** -10) + (0.0 if dtype != F32 else 2.0 ** -149)


def case(T, V, K, dtype, seed, ids_type=torch.int32, tdt=F32, ld=None):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * 2).to(dtype)
    ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(T)])
    teacher = (torch.randn(T, K, generator=g) + 2).to(tdt)
    ids[torch.rand(T, K, generator=g) < 0.2] = -1
    weight = torch.rand(T, generator=g)
    weight[torch.rand(T, generator=g) < 0.2] = 0
    if T > 3:
        ids[2] = -1  # nothing kept
        weight[1] = 0.5
    room = torch.zeros(T, ld or V, dtype=dtype, device="cuda")
    room[:, :V] = z.cuda()
    return room[:, :V], ids.to(ids_type).cuda(), teacher.cuda(), weight.cuda()


def check(z, ids, teacher, weight, tau=1.0, scale=1.0, in_place=False, grad=None, plan=None, S=1.0):
    h = [v.double().cpu().numpy() for v in (z, teacher, weight)]
    want_l, want_g, onto = formula(h[0], ids.cpu().numpy(), h[1], h[2], tau, scale * S)
    loss = torch.full((z.shape[0],), 7.0, device="cuda")
    out = z if in_place else torch.empty_like(z) if grad is None else grad
    zr.distill_topk(z, ids, teacher, loss, out, weight=weight, temperature=tau, grad_scale=scale, plan=plan)
    bl, bg = bounds(h[0], h[1], want_l, want_g, onto, h[2], tau, scale * S, z.dtype)
    dl, dg = np.abs(loss.double().cpu().numpy() - want_l), np.abs(out.double().cpu().numpy() - want_g)
    assert (dl <= bl).all(), (dl - bl).max()
    assert (dg <= bg).all(), ((dg - bg).max(), dg.max())
    return loss, out


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (1, 7, 3), (5, 8, 8), (9, 33, 4), (7, 1000, 17), (3, 5001, 100), (40, 4096, 64), (2, 50257, 256)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_loss_and_gradient(T, V, K, dtype):
    for i, tau in enumerate((1.0, 2.0, 0.5)):
        check(*case(T, V, K, dtype, seed=T + V + i, ids_type=(torch.int32, torch.int64)[i % 2], tdt=(F32, BF16, F16)[i]), tau=tau, scale=3.0)


@pytest.mark.parametrize("centre,tau,V", [(5000.0, 0.01, 900), (7000.0, 0.01, 900), (6931.0, 0.01, 60_000), (-3e4, 1e-3, 500), (1e30, 1.0, 300)])
def test_logits_far_from_zero_at_low_temperatures(centre, tau, V):
    """Exponents whose common part is from 10^5 to 10^30: only the differences count. The spread, not the magnitude,
    decides what fp32 may cost: the differences are exact up to two roundings of an exponent of at most A."""
    g = torch.Generator().manual_seed(V)
    ulp = float(np.spacing(np.float32(abs(centre))))
    z = (centre + max(ulp, tau) * torch.randint(-6, 7, (6, V), generator=g).double()).float().cuda()
    ids = torch.stack([torch.randperm(V, generator=g)[:9] for _ in range(6)]).int().cuda()
    teacher = (tau * torch.randn(6, 9, generator=g)).cuda()
    weight, loss, grad = torch.ones(6, device="cuda"), torch.empty(6, device="cuda"), torch.empty_like(z)
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight, temperature=tau)
    h = [v.double().cpu().numpy() for v in (z, teacher, weight)]
    l, want, onto = formula(h[0], ids.cpu().numpy(), h[1], h[2], tau, 1.0)
    spread = (h[0].max(1) - h[0].min(1)).max()
    bl, bg = bounds(h[0] - h[0].max(1, keepdims=True), h[1], l, want, onto, h[2], tau, 1.0, F32)
    assert spread > 0
    assert (np.abs(loss.double().cpu().numpy() - l) <= bl).all()
    assert (np.abs(grad.double().cpu().numpy() - want) <= bg).all()


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 logits: the last rows against the formula."""
    T, V, K = 44_000, 50_304, 4
    z = torch.empty(T, V, dtype=BF16, device="cuda")
    assert z.numel() > 1 << 31
    some = torch.tensor([0, 21_000, T - 2, T - 1])
    z.normal_()
    ids = torch.randint(0, V, (T, K), dtype=torch.int64, device="cuda")
    teacher, loss = torch.randn(T, K, device="cuda"), torch.empty(T, device="cuda")
    h = [v[some.cuda()].double().cpu().numpy() for v in (z, teacher)]
    w = np.ones(len(some))
    l, g, onto = formula(h[0], ids[some.cuda()].cpu().numpy(), h[1], w, 1.0, 1.0)
    zr.distill_topk(z, ids, teacher, loss, z)
    bl, bg = bounds(h[0], h[1], l, g, onto, w, 1.0, 1.0, BF16)
    assert (np.abs(loss[some.cuda()].double().cpu().numpy() - l) <= bl).all()
    assert (np.abs(z[some.cuda()].double().cpu().numpy() - g) <= bg).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_rows_and_long_rows(dtype):
    check(*case(400, 2000, 8, dtype, seed=1))       # a block for each row, several waves
    check(*case(1, 300_000, 30, dtype, seed=2))     # a row for a cluster
    check(*case(1, 600_001, 30, dtype, seed=3))     # more than a cluster's shared memory in 32 bits


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ldz,ldg", [(1003, 1003), (1003, 1001), (1008, 1003), (1001, 1008)])
def test_row_strides(dtype, ldz, ldg):
    z, ids, teacher, weight = case(12, 1001, 20, dtype, seed=ldz, ld=ldz)
    room = torch.full((12, ldg), 7.0, dtype=dtype, device="cuda")
    check(z, ids, teacher, weight, grad=room[:, :1001])
    assert bool((room[:, 1001:] == 7.0).all())


@pytest.mark.parametrize("V", [1000, 1001, 60_000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_gradient_over_the_logits(V, dtype):
    check(*case(6, V, 30, dtype, seed=V), in_place=True, scale=2.0)


def test_gradient_over_the_logits_longer_than_shared_memory():
    check(*case(1, 600_001, 30, F32, seed=3), in_place=True)


def test_repeated_entries():
    z, ids, teacher, weight = case(8, 500, 60, F32, seed=4)
    ids = ids % 7  # each column many times, in no order
    check(z, ids, teacher, weight)


def test_masked_logits_and_entries():
    """Vocabulary masked with -inf and with the type's lowest value, teacher entries of -inf, a row of only those."""
    z, ids, teacher, weight = case(8, 300, 10, BF16, seed=5)
    weight[:] = 1.0
    ids = ids.clamp(min=0) % 200
    z[:, 250:] = float("-inf")
    z[:, 200:250] = torch.finfo(BF16).min
    teacher[:, 3] = float("-inf")
    teacher[4] = float("-inf")
    loss, grad = check(z, ids, teacher, weight)
    assert float(loss[4]) == 0 and bool((grad[4] == 0).all()) and bool((grad[:, 250:] == 0).all())


def test_rows_without_loss_ignore_their_logits():
    z, ids, teacher, weight = case(6, 130, 5, F32, seed=6)
    weight[:] = 1.0
    weight[0], ids[1] = 0, -1
    z[0], z[1] = float("nan"), float("inf")
    check_rows = torch.tensor([0, 1])
    loss, grad = torch.empty(6, device="cuda"), torch.full_like(z, 7.0)
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight)
    assert bool((loss[check_rows] == 0).all()) and bool((grad[check_rows] == 0).all())
    assert bool(torch.isfinite(grad).all())


def test_rows_that_have_no_answer_say_so():
    """NaN, +inf, every logit masked, an id past the vocabulary, a NaN of the teacher: NaN in that row alone."""
    for V in (130, 50_000):
        z, ids, teacher, weight = case(8, V, 5, F32, seed=7)
        weight[:] = 1.0
        ids = ids.clamp(min=0)
        z[0, V - 1], z[1, 3], z[2] = float("nan"), float("inf"), float("-inf")
        ids[3, 2] = V
        loss, grad = torch.empty(8, device="cuda"), torch.empty_like(z)
        zr.distill_topk(z, ids, teacher, loss, grad, weight=weight)
        assert torch.equal(torch.isnan(loss).cpu(), torch.arange(8) < 4)
        assert torch.equal(torch.isnan(grad).any(1).cpu(), torch.arange(8) < 4)
        teacher[5, 0] = float("nan")
        zr.distill_topk(z, ids, teacher, loss, grad, weight=weight)
        assert bool(torch.isnan(loss[5])) and bool(torch.isnan(grad[5]).any()) and bool(torch.isfinite(loss[6]))


def test_loss_alone_and_no_weight():
    z, ids, teacher, _ = case(9, 700, 12, BF16, seed=8)
    one, two = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    zr.distill_topk(z, ids, teacher, one, temperature=2.0)
    zr.distill_topk(z, ids, teacher, two, torch.empty_like(z), weight=torch.ones(9, device="cuda"), temperature=2.0)
    assert torch.equal(one, two)


def test_gradient_against_differences():
    """Central differences of the loss. The formula's third derivative is under w/tau, so a step of 1/8 costs under
    h^2/6; the losses' fp32 errors cost 2 * bound / (2 h)."""
    z, ids, teacher, weight = case(4, 40, 6, F32, seed=9)
    weight[:] = 1.0
    tau, h = 1.5, 0.125
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(z)
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight, temperature=tau)
    hz = [v.double().cpu().numpy() for v in (z, teacher, weight)]
    l, g, onto = formula(hz[0], ids.cpu().numpy(), hz[1], hz[2], tau, 1.0)
    bl = bounds(hz[0], hz[1], l, g, onto, hz[2], tau, 1.0, F32)[0].max()
    up, down = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    for v in range(0, 40, 3):
        step = torch.zeros_like(z)
        step[:, v] = h
        zr.distill_topk(z + step, ids, teacher, up, weight=weight, temperature=tau)
        zr.distill_topk(z - step, ids, teacher, down, weight=weight, temperature=tau)
        d = ((up - down).double() / (2 * h)).cpu().numpy()
        assert (np.abs(d - grad[:, v].double().cpu().numpy()) <= h * h / 6 + 2 * bl / h + 1e-6).all()


def test_plan_scales_the_gradient():
    """The plan's loss scale is read on the device: after a skipped step the same captured call uses the halved one."""
    plan = zr.Plan([64], W=1, dtype=zr.F16, stage=1, cap=64, scaler=zr.Scaler(init_scale=1024.0, dynamic=True))
    z, ids, teacher, weight = case(5, 64, 4, F32, seed=10)
    check(z, ids, teacher, weight, plan=plan, S=1024.0, scale=0.5)
    loss, grad = torch.empty(5, device="cuda"), torch.empty_like(z)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        zr.distill_topk(z, ids, teacher, loss, grad, weight=weight, plan=plan, stream=side)
    graph.replay()
    before = grad.clone()
    state = plan.new_state()
    for k in range(2):
        state.master[k].zero_(), state.param[k].zero_()
    rep = plan.step([torch.full((64,), float("inf"), dtype=F16, device="cuda")], state, zr.AdamW(), report=True)
    assert rep.skipped == 1 and rep.scale == 512.0
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad * 2, before)


def test_what_does_not_fit_is_refused():
    z, ids, teacher, weight = case(4, 50, 3, F32, seed=12)
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(z)
    ok = dict(logits=z, ids=ids, teacher=teacher, loss=loss, grad=grad, weight=weight)
    for bad in (dict(ids=ids.short()), dict(ids=ids[:, :2]), dict(ids=ids[:3], teacher=teacher[:3]), dict(ids=ids.cpu()),
                dict(loss=loss[:3]), dict(loss=loss.double()), dict(weight=weight[:3]), dict(grad=grad.half()),
                dict(grad=grad[:, :49]), dict(logits=z.double(), grad=grad.double()), dict(temperature=0.0),
                dict(grad_scale=float("inf")), dict(ids=ids.t().contiguous().t()), dict(teacher=teacher.t().contiguous().t()),
                dict(logits=z[:, 1:], grad=grad[:, 1:])):
        with pytest.raises(zr.ZrError) as e:
            zr.distill_topk(**{**ok, **bad})
        assert e.value.status == 1, bad
    zr.distill_topk(**ok)


def test_other_stream_and_guards():
    z, ids, teacher, weight = case(7, 999, 12, BF16, seed=11)
    raw = torch.full((7 * 999 + 2048,), 7.0, dtype=BF16, device="cuda")
    grad, loss = raw[1024:1024 + 7 * 999].view(7, 999), torch.empty(7, device="cuda")
    ref_loss, ref_grad = check(z, ids, teacher, weight)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    zr.distill_topk(z, ids, teacher, loss, grad, weight=weight, stream=side)
    side.synchronize()
    assert torch.equal(loss, ref_loss) and torch.equal(grad, ref_grad)
    assert bool((raw[:1024] == 7).all()) and bool((raw[1024 + 7 * 999:] == 7).all())


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,V,dtype", [(160, 58_001, BF16), (160, 29_000, F32), (155, 121_000, F16), (154, 62_003, F32)])
def test_rows_that_shared_memory_holds_a_part_of(T, V, dtype, in_place):
    """A block's, and a cluster's blocks': more rows than multiprocessors, each a little over what is kept of it. What is
    read again adds, for each thread, under ten sums of four words and as many changes of its maximum."""
    check(*case(T, V, 20, dtype, seed=V), tau=2.0, in_place=in_place)


@pytest.mark.parametrize("K,columns", [(1024, 1), (1024, 700), (300, 5), (33, 16)])
def test_columns_that_stand_many_times(K, columns):
    z, ids, teacher, weight = case(9, 3000, K, BF16, seed=K + columns)
    keep = ids < 0
    ids = torch.where(keep, ids, 2990 - ids % columns * 4)
    check(z, ids, teacher, weight)


def test_the_largest_logit_in_the_part_that_is_read_again():
    """Its sum is relative to its own maximum, which the part kept in shared memory comes to take over, and the other way round."""
    z, ids, teacher, weight = case(160, 58_000, 20, BF16, seed=5)
    z[::2, -1] = 60.0
    z[1::2, 0] = 60.0
    z[::3, -3000:] = -float("inf")
    z[1::3, :40_000] = -float("inf")
    ids[(ids < 40_000) | (ids > 54_000)] = -1
    z[:, 45_000] = 1.0
    ids[:, 0] = 45_000
    check(z, ids, teacher, weight)
