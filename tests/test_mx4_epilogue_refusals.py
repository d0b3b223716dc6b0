"""What the products with an epilogue and the column sums refuse, before any CUDA call and so without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import zero_gradient_reduction_gb300 as zr  # noqa: E402
from test_losses_refusals import Vector  # noqa: E402
from test_mx4_devices import Tensor, mx4  # noqa: E402
from test_mx4_refusals import L, refused  # noqa: E402,F401  (L: the built library)

M, N, K = 4, 8, 32
OUT = 1 << 20


def epilogue(**fields):
    e = zr.Epilogue()
    e.ldr = e.ldp = N
    for k, v in fields.items():
        setattr(e, k, v)
    return e


def matmul(L, e, a=16, out=OUT, dt=2, ldo=N, m=M):
    return L.zr_mx4_matmul_finish(a, m, 16, N, K, out, dt, ldo, ctypes.byref(e) if e else None, None)


def linear(L, e, a=16, out=OUT, dt=2, ldo=N, m=M):
    return L.zr_mx4_linear_finish(a, 2, m, K, 16, N, K, out, dt, ldo, None, ctypes.byref(e) if e else None, None)


@pytest.mark.parametrize("call", [matmul, linear])
def test_epilogues(L, call):
    for bad in (-1, 4):
        refused(L, call(L, epilogue(activation=bad)), "activation")
    refused(L, call(L, epilogue(bias=16, bias_dtype=5)), "dtype")
    refused(L, call(L, epilogue(pre=1 << 22, ldp=N - 1)), "stride")
    refused(L, call(L, epilogue(residual=1 << 22, ldr=N - 1)), "stride")
    refused(L, call(L, epilogue(gradient=1)), "gradient")
    refused(L, call(L, epilogue(gradient=1, pre=1 << 22, bias=16)), "gradient")
    refused(L, call(L, epilogue(gradient=1, pre=1 << 22, residual=1 << 23)), "gradient")
    for name in ("bias", "pre", "residual"):
        refused(L, call(L, epilogue(**{name: (1 << 22) + 8}, bias_dtype=2)), "aligned")
    # out, pre and residual share memory
    refused(L, call(L, epilogue(pre=OUT)), "overlap")
    refused(L, call(L, epilogue(pre=OUT + 16)), "overlap")
    refused(L, call(L, epilogue(residual=OUT + 16)), "overlap")
    refused(L, call(L, epilogue(residual=OUT, ldr=N + 4)), "overlap")
    refused(L, call(L, epilogue(residual=1 << 22, pre=1 << 22)), "overlap")
    refused(L, call(L, epilogue(gradient=1, pre=OUT + 16)), "overlap")
    refused(L, call(L, epilogue(residual=OUT + (2 * N - 4) * 4, ldr=2 * N), ldo=2 * N), "overlap")
    # what they refuse without one
    refused(L, call(L, epilogue(), dt=7), "dtype")
    refused(L, call(L, epilogue(), ldo=N - 1), "stride")
    refused(L, call(L, epilogue(), a=None), "null")
    refused(L, call(L, epilogue(), a=24), "aligned")
    refused(L, call(L, None, a=None), "null")
    assert call(L, epilogue(), m=0, a=None) == 0


def test_tokens_in_the_place_of_results(L):
    """x as the residual and the output of one call: few tokens would be read after other blocks had replaced them."""
    refused(L, linear(L, epilogue(residual=OUT), a=OUT), "overlaps x")
    refused(L, linear(L, epilogue(), a=OUT + 16), "overlaps x")
    refused(L, linear(L, epilogue(pre=1 << 22), a=(1 << 22) - 16), "overlaps x")
    # rows of 32 bytes of out between rows of 128 bytes of tokens (no weights then), and too near to either end
    def between(out):
        return L.zr_mx4_linear_finish(OUT, 2, M, 40, None, N, K, out, 2, 40, None, ctypes.byref(epilogue()), None)
    refused(L, between(OUT + 128), "null")
    refused(L, between(OUT + 112), "overlaps x")
    refused(L, between(OUT + 144), "overlaps x")


def test_column_sums(L):
    c = L.zr_column_sums
    refused(L, c(16, 7, 4, 8, 8, 16, None), "dtype")
    refused(L, c(16, 2, -1, 8, 8, 16, None), "negative")
    refused(L, c(16, 2, 4, 8, 7, 16, None), "stride")
    refused(L, c(None, 2, 4, 8, 8, 16, None), "null")
    refused(L, c(16, 2, 4, 8, 8, None, None), "null")
    refused(L, c(24, 2, 4, 8, 8, 16, None), "aligned")
    refused(L, c(16, 2, 4, 8, 8, 18, None), "aligned")
    assert c(None, 2, 4, 0, 0, None, None) == 0


@pytest.fixture
def calls(monkeypatch, L):
    made = []
    monkeypatch.setattr(zr, "_fns", {
        "stream": lambda device: 0, "device": lambda: 0, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64,
        **{name: (lambda *a, n=name: made.append((n, a)) or 0) for name in (
            "zr_mx4_matmul", "zr_mx4_linear", "zr_mx4_matmul_finish", "zr_mx4_linear_finish", "zr_column_sums")}})
    monkeypatch.setattr(zr, "_types", {torch.float16: zr.F16, torch.bfloat16: zr.BF16, torch.float32: zr.F32})
    return made


def operands(call):
    own = dict(out=lambda d: Tensor((M, N), device=d), bias=lambda d: Vector((N,), device=d), residual=lambda d: Tensor((M, N), device=d),
               pre=lambda d: Tensor((M, N), device=d))
    if call == "matmul":
        return zr.mx4_matmul, dict(a=lambda d: mx4(M, K, d), b=lambda d: mx4(N, K, d), **own)
    return zr.mx4_linear, dict(x=lambda d: Tensor((M, K), device=d), w=lambda d: mx4(N, K, d), **own)


@pytest.mark.parametrize("call", ["matmul", "linear"])
def test_the_binding(calls, call):
    fn, makers = operands(call)
    good = {k: make(0) for k, make in makers.items()}
    fn(**good, activation="gelu")
    assert calls.pop()[0] == f"zr_mx4_{call}_finish"
    fn(**{k: v for k, v in good.items() if k not in ("bias", "residual", "pre")})
    assert calls.pop()[0] == f"zr_mx4_{call}"
    for name in makers:
        with pytest.raises(zr.ZrError) as e:
            fn(**{**good, name: makers[name](1)})
        assert e.value.status == 1 and "device" in str(e.value) and not calls
    for bad in (dict(activation="tanh"), dict(bias=Vector((N + 1,))), dict(bias=Vector((N,), torch.float64)), dict(bias=Vector((N,), device=-1)),
                dict(pre=Tensor((M, N + 1))), dict(pre=Tensor((M, N), torch.float16)), dict(residual=Tensor((M + 1, N))),
                dict(residual=Tensor((M, N), torch.bfloat16))):
        with pytest.raises(zr.ZrError):
            fn(**{**good, **bad})
    assert not calls


def test_the_epilogue_that_the_binding_passes(calls):
    fn, makers = operands("matmul")
    good = {k: make(0) for k, make in makers.items()}
    fn(**good, activation="silu")
    e = zr.Epilogue.from_buffer_copy(calls.pop()[1][8])
    assert (e.bias, e.residual, e.pre, e.ldr, e.ldp, e.activation, e.gradient) == (*(good[k].data_ptr() for k in ("bias", "residual", "pre")), N, N, 3, 0)
    assert e.bias_dtype == zr._types[good["bias"].dtype]
    fn(good["a"], good["b"], good["out"], gradient_of="relu", pre=good["pre"])
    e = zr.Epilogue.from_buffer_copy(calls.pop()[1][8])
    assert (e.bias, e.residual, e.pre, e.ldr, e.ldp, e.activation, e.gradient) == (None, None, good["pre"].data_ptr(), 0, N, 1, 1)


def test_a_gradient_of_no_rows(calls):
    """Matrices without values have no address, which would read as a gradient without pre."""
    zr.mx4_matmul(mx4(0, K, 0), mx4(N, K, 0), Tensor((0, N)), gradient_of="relu", pre=Tensor((0, N)))
    assert not calls


def test_what_the_binding_packs_is_what_the_library_reads(L):
    packed = zr._pack_epilogue(0, 0, 0, N, N, 2, 4, 0)
    refused(L, L.zr_mx4_matmul_finish(16, M, 16, N, K, OUT, 2, N, packed, None), "activation 4")
    refused(L, L.zr_mx4_matmul_finish(16, M, 16, N, K, OUT, 2, N, zr._pack_epilogue(0, 0, OUT + 16, 0, N, 2, 1, 1), None), "overlap")


def test_gradients_through_the_binding(calls):
    fn, makers = operands("matmul")
    good = {k: makers[k](0) for k in ("a", "b", "out", "pre")}
    fn(**good, gradient_of="relu")
    assert calls.pop()[0] == "zr_mx4_matmul_finish"
    for bad in (dict(gradient_of="relu", activation="relu"), dict(gradient_of="tanh")):
        with pytest.raises(zr.ZrError):
            fn(**good, **bad)
    assert not calls


def test_column_sums_through_the_binding(calls):
    zr.column_sums(Tensor((M, N)), Vector((N,)))
    assert calls.pop()[0] == "zr_column_sums"
    for out in (None, Vector((N + 1,)), Vector((N,), torch.float16), Vector((N,), device=1), Vector((N,), device=-1)):
        with pytest.raises(zr.ZrError):
            zr.column_sums(Tensor((M, N)), out)
    assert not calls
