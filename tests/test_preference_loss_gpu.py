"""The loss of pairs of sequences by their log-probability ratios, and its gradient, against the formulas in 64 bits."""
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


def workspace(T, pairs, fill=255):
    return torch.full((zr.preference_bytes(T, pairs),), fill, dtype=torch.uint8, device="cuda")


def case(lengths, V, dtype, seed, tau=1.0, before=0, behind=0, ld=None):
    """(logits, ids, starts, reference, weights) of sequences of these lengths, with rows of no sequence around them."""
    g = torch.Generator().manual_seed(seed)
    starts = before + np.concatenate([[0], np.cumsum(lengths)])
    T = int(starts[-1]) + behind
    z, ids = ref.logits(T, V, dtype, g, ld=ld)
    logp = ref.softmax(host(z), tau)[0][np.arange(T), ids.numpy()]
    near_ref = torch.from_numpy(logp + 0.5 * torch.randn(T, generator=g).double().numpy()).float().cuda()
    ids[torch.rand(T, generator=g) < 0.2] = -1
    return z, ids, torch.from_numpy(starts), near_ref, (torch.rand(len(lengths) // 2, generator=g) + 0.2).cuda()


def check(z, ids, starts, near_ref, weight, beta=0.3, smoothing=0.1, tau=1.0, scale=1.0, grad=None, in_place=False, plan=None, S=1.0,
          ids_type=torch.int64, starts_type=torch.int32):
    T, pairs = z.shape[0], len(weight)
    h, a = host(z), ids.numpy()
    (loss, rewards, f, inside), (e_loss, e_rewards, e_f) = ref.preference(
        h, a, starts.numpy(), host(near_ref), host(weight), float(np.float32(beta)), float(np.float32(smoothing)), tau, scale * S)
    out = z if in_place else torch.full_like(z, 7.0) if grad is None else grad
    was = out.clone()
    got, r = torch.full((pairs,), 7.0, device="cuda"), torch.full((2 * pairs,), 7.0, device="cuda")
    zr.preference_loss(z, ids.to(ids_type).cuda(), starts.to(starts_type).cuda(), near_ref, got, workspace(T, pairs), out, weight=weight,
                       beta=beta, smoothing=smoothing, rewards=r, temperature=tau, grad_scale=scale, plan=plan)
    near(r, rewards, e_rewards, "rewards")
    near(got, loss, e_loss, "loss")
    at, inside = np.maximum(a, 0), torch.from_numpy(inside)
    near(out[inside.cuda()], ref.gradient(h, tau, at, f)[inside], ref.gradient_error(h, tau, at, f, e_f, z.dtype)[inside], "gradient")
    assert torch.equal(out[~inside.cuda()], was[~inside.cuda()])
    return got, r, out


@pytest.mark.parametrize("lengths", [(1, 1), (0, 3), (2, 0), (0, 0), (5, 9, 4, 1), (40, 33, 1, 70, 0, 0, 13, 2), tuple([3, 2] * 40)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_loss_and_gradient(lengths, dtype):
    for i, (V, beta, smoothing) in enumerate(((33, 0.1, 0.0), (1001, 0.5, 0.1), (1000, 2.0, 0.5))):
        check(*case(lengths, V, dtype, seed=len(lengths) + i, before=i, behind=2 * i), beta=beta, smoothing=smoothing, scale=3.0,
              ids_type=(torch.int64, torch.int32)[i % 2], starts_type=(torch.int32, torch.int64)[i % 2])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_and_many_rows(dtype):
    check(*case((2, 3), 50257, dtype, seed=1))           # a row for a cluster
    check(*case((1, 1), 600_001, dtype, seed=2))
    check(*case((700, 650, 20, 900), 500, dtype, seed=3))  # several waves


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ldz,ldg", [(1003, 1003), (1003, 1001), (1008, 1003), (1001, 1008)])
def test_row_strides(dtype, ldz, ldg):
    room = torch.full((17, ldg), 7.0, dtype=dtype, device="cuda")
    check(*case((5, 6, 4, 2), 1001, dtype, seed=ldz, ld=ldz), grad=room[:, :1001])
    assert bool((room[:, 1001:] == 7.0).all())


@pytest.mark.parametrize("at", [0, 1, 7, 8, 9, 500, 1000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_each_place_in_a_row(dtype, at):
    z, ids, *rest = case((5, 4), 1001, dtype, seed=at, ld=1003)
    check(z, torch.where(ids < 0, ids, at), *rest)


@pytest.mark.parametrize("V", [1000, 1001, 60_000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_gradient_over_the_logits(V, dtype):
    check(*case((4, 3), V, dtype, seed=V, before=1, behind=1), in_place=True, scale=2.0)


def test_long_sequences():
    """Thousands of rows a sequence: the sums of their ratios, and margins far out on both sides."""
    z, ids, starts, near_ref, weight = case((3000, 2500, 2600, 3100), 65, F32, seed=4)
    for beta in (0.01, 1.0):
        check(z, ids, starts, near_ref, weight, beta=beta, smoothing=0.0)


def test_a_pair_without_weight_is_not_read():
    z, ids, starts, near_ref, weight = case((4, 5, 3, 2), 130, F32, seed=5)
    ids = ids.clamp(min=0)
    weight[0] = 0
    z[:9], near_ref[:9] = NAN, NAN
    loss, r, grad = torch.empty(2, device="cuda"), torch.empty(4, device="cuda"), torch.full_like(z, 7.0)
    zr.preference_loss(z, ids.cuda(), starts.cuda(), near_ref, loss, workspace(14, 2), grad, weight=weight, rewards=r)
    assert float(loss[0]) == 0 and float(loss[1]) > 0 and bool((r[:2] == 0).all()) and bool((grad[:9] == 0).all())
    assert bool(torch.isfinite(grad).all()) and bool((grad[9:] != 0).any())


def test_rows_that_have_no_answer_say_so_in_their_pair():
    for V in (130, 50_000):
        z, ids, starts, near_ref, weight = case((3, 2) * 12, V, F32, seed=6, behind=1)
        starts = starts[:13]
        z, ids, near_ref = z[:31], ids[:31].clamp(min=0), near_ref[:31].contiguous()
        ids[4::5] = -1  # the last row of each pair is not scored
        z[0, V - 1], z[5, 3], z[10] = NAN, INF, -INF
        ids[15] = V
        near_ref[20] = NAN
        z[29], near_ref[29] = NAN, NAN  # not scored
        z[30] = NAN                     # of no sequence
        loss, r, grad = torch.empty(6, device="cuda"), torch.empty(12, device="cuda"), torch.full_like(z, 7.0)
        zr.preference_loss(z, ids.cuda(), starts.cuda(), near_ref, loss, workspace(31, 6), grad, rewards=r)
        assert torch.isnan(loss).tolist() == [True] * 5 + [False]
        assert torch.isnan(r).tolist() == [True, False] * 5 + [False, False]
        bad = torch.tensor([i < 25 and i % 5 != 4 for i in range(31)])
        assert torch.equal(torch.isnan(grad).all(1).cpu(), bad) and not bool(torch.isnan(grad[~bad.cuda()]).any())
        assert bool((grad[30] == 7.0).all()) and bool((grad[4:30:5] == 0).all())


def test_a_masked_token_in_a_sequence():
    """logp = -inf on one side: an infinite margin, whose loss is infinite or nothing, and no gradient that is no number."""
    z, ids, starts, near_ref, weight = case((3, 2, 3, 2), 50, F32, seed=7)
    ids = ids.clamp(min=0, max=40)
    ids[1] = ids[8] = 45
    z[:, 45] = -INF
    loss, grad = torch.empty(2, device="cuda"), torch.empty_like(z)
    zr.preference_loss(z, ids.cuda(), starts.cuda(), near_ref, loss, workspace(10, 2), grad)
    assert loss.tolist() == [INF, 0.0] and bool(torch.isfinite(grad).all())
    assert float(grad[1, 45]) < 0 and bool((grad[5:] == 0).all())


def test_starts_that_do_not_ascend():
    """No row outside the arrays is read or written, and the pairs that are wrong say so."""
    T, V = 12, 40
    z, ids = ref.logits(T, V, F32, torch.Generator().manual_seed(8))
    for starts, bad in (((0, 3, 2, 5, 12), [True, False]), ((0, 3, 6, 9, 13), [False, True]), ((-1, 3, 6, 9, 12), [True, False]),
                        ((0, 1 << 40, 6, 9, 12), [True, False]), ((-(1 << 62), 1 << 62, -5, 3, 2), [True, True])):
        room = torch.full((T + 2, V), 7.0, device="cuda")
        loss = torch.empty(2, device="cuda")
        guard = torch.full((zr.preference_bytes(T, 2) + 64,), 77, dtype=torch.uint8, device="cuda")
        zr.preference_loss(z, ids.cuda(), torch.tensor(starts, device="cuda"), torch.zeros(T, device="cuda"), loss, guard[:-64], room[1:-1])
        assert torch.isnan(loss).tolist() == bad, starts
        assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all()) and bool((guard[-64:] == 77).all())


def test_gradient_against_differences():
    lengths, V, h = (2, 3, 1, 2), 7, 1e-5
    z, ids, starts, near_ref, weight = case(lengths, V, F32, seed=9, tau=1.3)
    ids = ids.clamp(min=0)
    ids[3] = -1
    loss, grad = torch.empty(2, device="cuda"), torch.empty_like(z)
    zr.preference_loss(z, ids.cuda(), starts.cuda(), near_ref, loss, workspace(8, 2), grad, weight=weight, beta=0.7, smoothing=0.2, temperature=1.3)
    x = host(z)

    def total(y):
        return ref.preference(y, ids.numpy(), starts.numpy(), host(near_ref), host(weight), float(np.float32(0.7)), float(np.float32(0.2)), 1.3, 1.0)[0][0].sum()

    for t in range(8):
        for v in range(V):
            up, down = x.copy(), x.copy()
            up[t, v] += h
            down[t, v] -= h
            slope = (total(up) - total(down)) / (2 * h)
            assert abs(float(grad[t, v]) - slope) <= 1e-4 * np.abs(host(grad)).max() + 1e-8


def test_the_plans_loss_scale():
    plan = zr.Plan([64], W=1, dtype=zr.F16, stage=1, cap=64, scaler=zr.Scaler(init_scale=512.0))
    check(*case((4, 3), 100, F32, seed=10), plan=plan, scale=2.0, S=512.0)
    plan.close()


def test_captured_twice_and_at_once():
    """Two captured passes with a workspace each, replayed at the same time on two streams, and replayed on other
    sequences: the bytes of plain calls."""
    z, ids, starts, near_ref, weight = case((30, 41, 22, 7), 2000, BF16, seed=11)
    ids, starts = ids.cuda(), starts.int().cuda()

    def outputs():
        return [torch.empty(2, device="cuda"), torch.full_like(z, 7.0), workspace(100, 2)]

    def call(o, k):
        zr.preference_loss(z, ids, starts, near_ref, o[0], o[2], o[1], weight=weight, beta=0.1 + k)

    outs, graphs = [], []
    for k in range(2):
        o = outputs()
        call(o, k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                call(o, k)
        outs.append(o)
        graphs.append(graph)
    for bounds in ((0, 30, 71, 93, 100), (5, 40, 41, 90, 95)):
        starts.copy_(torch.tensor(bounds, dtype=torch.int32))
        want = []
        for k in range(2):
            o = outputs()
            call(o, k)
            want.append(o)
            outs[k][1].fill_(7.0)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k][0], want[k][0]) and torch.equal(outs[k][1], want[k][1])


def test_no_pairs_and_no_rows():
    z = torch.full((3, 50), 2.0, device="cuda")
    ids, grad = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.full_like(z, 7.0)
    zr.preference_loss(z, ids, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda"), torch.empty(0, device="cuda"),
                       workspace(3, 0), grad)
    assert bool((grad == 7.0).all())
    loss, r = torch.empty(2, device="cuda"), torch.empty(4, device="cuda")
    zr.preference_loss(z[:0], ids[:0], torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda"), loss, workspace(0, 2),
                       grad[:0], rewards=r)
    assert np.allclose(loss.cpu().numpy(), np.log(2.0), rtol=1e-6) and bool((r == 0).all())


@pytest.mark.parametrize("pairs,rows", [(1, 700), (2, 3000), (700, 2), (40, 60), (3, 1)])
def test_rows_of_many_shapes_in_order(pairs, rows):
    """Few long and many short pairs, empty ones among them, on rows that go in parts and in whole: more blocks than run at once."""
    g = torch.Generator().manual_seed(pairs)
    lengths = torch.randint(0, 2 * rows, (2 * pairs,), generator=g).tolist()
    check(*case(lengths, 120, BF16, seed=pairs, before=3, behind=2))
    check(*case([min(n, 3) for n in lengths[:20]], 40_000, BF16, seed=pairs))
