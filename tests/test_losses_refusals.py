"""Arguments that the post-training losses refuse, before any CUDA call and so without a GPU."""
import types

import pytest

torch = pytest.importorskip("torch")
import zero_gradient_reduction_gb300 as zr  # noqa: E402
from test_mx4_devices import Tensor  # noqa: E402
from test_mx4_refusals import L, refused  # noqa: E402,F401  (L: the built library)

NAN, INF = float("nan"), float("inf")


def logprobs(L, z=16, dt=2, T=4, V=50, ldz=50, ids=16, wide=0, tau=1.0, logp=16, entropy=None):
    return L.zr_token_logprobs(z, dt, T, V, ldz, ids, wide, tau, logp, entropy, None)


def policy(L, z=16, dt=2, T=4, V=50, ldz=50, ids=16, wide=0, old=16, adv=16, w=16, lo=0.2, hi=0.2, ref=16, kl=0.1, tau=1.0, scale=1.0,
           loss=16, logp=16, grad=1 << 20, ldg=50):
    return L.zr_policy_loss(z, dt, T, V, ldz, ids, wide, old, adv, w, lo, hi, ref, kl, tau, scale, None, loss, logp, grad, ldg, None)


def preference(L, z=16, dt=2, T=4, V=50, ldz=50, ids=16, wide=0, starts=16, wide_starts=0, pairs=1, ref=16, w=16, beta=0.1, smoothing=0.0,
               tau=1.0, scale=1.0, loss=16, rewards=16, grad=1 << 20, ldg=50, work=16):
    return L.zr_preference_loss(z, dt, T, V, ldz, ids, wide, starts, wide_starts, pairs, ref, w, beta, smoothing, tau, scale, None, loss, rewards,
                                grad, ldg, work, None)


@pytest.mark.parametrize("call", [logprobs, policy, preference])
def test_what_all_refuse(L, call):
    refused(L, call(L, dt=7), "dtype")
    refused(L, call(L, T=-1), "T must")
    for V in (0, -5, 1 << 31):
        refused(L, call(L, V=V, ldz=1 << 32), "V in")
    refused(L, call(L, ldz=49), "stride")
    for tau in (0.0, -1.0, NAN, INF, 1e-7):
        refused(L, call(L, tau=tau), "temperature")
    refused(L, call(L, z=None), "null")
    refused(L, call(L, ids=None), "null")
    refused(L, call(L, z=24), "aligned")
    refused(L, call(L, ids=18), "aligned")
    refused(L, call(L, ids=20, wide=1), "aligned")


def test_logprobs(L):
    refused(L, logprobs(L, logp=None), "null")
    refused(L, logprobs(L, logp=18), "aligned")
    refused(L, logprobs(L, entropy=18), "aligned")
    assert logprobs(L, T=0, z=None) == 0


def test_policy(L):
    for lo, hi in ((-0.1, 0.2), (1.1, 0.2), (NAN, 0.2), (0.2, -0.1), (0.2, NAN), (0.2, INF)):
        refused(L, policy(L, lo=lo, hi=hi), "clip")
    refused(L, policy(L, kl=NAN), "kl")
    refused(L, policy(L, kl=0.1, ref=None), "ref_logp")
    refused(L, policy(L, scale=INF), "grad_scale")
    refused(L, policy(L, ldg=49), "stride")
    for name in ("old", "adv", "loss"):
        refused(L, policy(L, **{name: None}), "null")
    for name in ("old", "adv", "w", "ref", "loss", "logp"):
        refused(L, policy(L, **{name: 18}), "aligned")
    refused(L, policy(L, grad=(1 << 20) + 8), "aligned")
    refused(L, policy(L, z=1 << 20, grad=(1 << 20) + 16), "overlaps")
    refused(L, policy(L, z=1 << 20, grad=1 << 20, ldg=51), "overlaps")
    assert policy(L, T=0, z=None) == 0


def test_preference(L):
    refused(L, preference(L, pairs=-1), "pairs")
    refused(L, preference(L, beta=NAN), "beta")
    refused(L, preference(L, scale=INF), "grad_scale")
    for smoothing in (-0.1, 1.1, NAN):
        refused(L, preference(L, smoothing=smoothing), "smoothing")
    refused(L, preference(L, ldg=49), "stride")
    for name in ("starts", "ref", "loss", "work"):
        refused(L, preference(L, **{name: None}), "null")
    for name in ("ref", "w", "loss", "rewards", "starts"):
        refused(L, preference(L, **{name: 18}), "aligned")
    refused(L, preference(L, starts=20, wide_starts=1), "aligned")
    refused(L, preference(L, work=24), "aligned")
    refused(L, preference(L, z=1 << 20, grad=(1 << 20) + 16), "overlaps")
    assert preference(L, T=1 << 29, V=1, ldz=1) == 2
    assert preference(L, pairs=0, loss=None, starts=None) == 0
    assert L.zr_preference_bytes(-1, 2) == -1 and L.zr_preference_bytes(2, -1) == -1 and L.zr_preference_bytes(1 << 40, 1) == -1


# ------------------------------------------------------------------ through the binding
class Vector(Tensor):
    def stride(self):
        return (1,)


@pytest.fixture
def calls(monkeypatch, L):
    made = []
    monkeypatch.setattr(zr, "_fns", {"stream": lambda device: 0, "device": lambda: 0, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64,
                                     **{name: (lambda *a: made.append(a) or 0) for name in ("zr_token_logprobs", "zr_policy_loss", "zr_preference_loss")}})
    monkeypatch.setattr(zr, "_types", {torch.float16: zr.F16, torch.bfloat16: zr.BF16, torch.float32: zr.F32})
    return made


def operands(call):
    f32 = lambda n: lambda d, t=torch.float32: Vector((n,), t, d)  # noqa: E731
    whole = lambda n: lambda d, t=torch.int64: Vector((n,), t, d)  # noqa: E731
    z = dict(logits=lambda d: Tensor((4, 50), device=d), ids=whole(4))
    plan = lambda d: types.SimpleNamespace(handle=1, device=d)  # noqa: E731
    grad = lambda d: Tensor((4, 50), device=d)  # noqa: E731
    if call == "logprobs":
        return zr.token_logprobs, dict(**z, logp=f32(4), entropy=f32(4))
    if call == "policy":
        return zr.policy_loss, dict(**z, old_logp=f32(4), advantage=f32(4), loss=f32(4), grad=grad, weight=f32(4), ref_logp=f32(4), logp=f32(4), plan=plan)
    return zr.preference_loss, dict(**z, starts=whole(3), ref_logp=f32(4), loss=f32(1), work=lambda d: Vector((1 << 16,), torch.uint8, d), grad=grad,
                                    weight=f32(1), rewards=f32(2), plan=plan)


CALLS = ["logprobs", "policy", "preference"]


def made_on(makers, elsewhere=None):
    return {k: make(1 if k == elsewhere else 0) for k, make in makers.items()}


@pytest.mark.parametrize("call", CALLS)
def test_together_on_the_current_device(calls, call):
    fn, makers = operands(call)
    fn(**made_on(makers))
    assert len(calls) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in operands(c)[1]])
def test_one_operand_elsewhere(calls, call, name):
    fn, makers = operands(call)
    with pytest.raises(zr.ZrError) as e:
        fn(**made_on(makers, name))
    assert e.value.status == 1 and "device" in str(e.value) and not calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(calls, call):
    fn, makers = operands(call)
    fn(**made_on(makers), stream=types.SimpleNamespace(cuda_stream=64, device_index=0))
    assert calls.pop()[-1] == 64
    with pytest.raises(zr.ZrError):
        fn(**made_on(makers), stream=types.SimpleNamespace(cuda_stream=64, device_index=1))
    assert not calls


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in operands(c)[1] if n not in ("logits", "plan", "grad", "work")])
def test_vectors_of_other_sizes_and_types(calls, call, name):
    fn, makers = operands(call)
    whole = name in ("ids", "starts")
    good = makers[name](0)
    for bad in (Vector((7,), good.dtype), Vector(good.shape, torch.float16 if not whole else torch.int16), Vector(good.shape, good.dtype, device=-1)):
        with pytest.raises(zr.ZrError):
            fn(**{**made_on(makers), name: bad})
    strided = Vector(good.shape, good.dtype)
    strided.is_contiguous = lambda: False
    with pytest.raises(zr.ZrError):
        fn(**{**made_on(makers), name: strided})
    assert not calls


@pytest.mark.parametrize("rows,pairs", [(0, 1), (1, 1), (2, 1), (3, 2), (4, 7), (5, 2), (61, 1), (8192, 16), (1000, 999)])
def test_the_workspace_is_as_large_as_the_library_says(calls, rows, pairs):
    """A byte less is refused, by the same count."""
    need = zr.preference_bytes(rows, pairs)

    def call(size):
        zr.preference_loss(Tensor((rows, 50)), Vector((rows,), torch.int64), Vector((2 * pairs + 1,), torch.int64), Vector((rows,)), Vector((pairs,)),
                           Vector((size,), torch.uint8))

    call(need)
    assert len(calls) == 1
    if need:
        with pytest.raises(zr.ZrError) as e:
            call(need - 1)
        assert str(need) in str(e.value)


def test_other_refusals(calls):
    fn, makers = operands("preference")
    with pytest.raises(zr.ZrError):
        fn(**{**made_on(makers), "work": Vector((10,), torch.uint8)})
    for call in ("policy", "preference"):
        fn, makers = operands(call)
        for bad in (Tensor((4, 51)), Tensor((4, 50), torch.float16)):
            with pytest.raises(zr.ZrError):
                fn(**{**made_on(makers), "grad": bad})
    for call, name in (("logprobs", "logp"), ("policy", "loss"), ("policy", "old_logp"), ("policy", "advantage"), ("preference", "loss"),
                       ("preference", "ref_logp")):
        fn, makers = operands(call)
        with pytest.raises(zr.ZrError):
            fn(**{**made_on(makers), name: None})
    assert not calls
