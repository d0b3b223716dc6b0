"""Operands that do not lie together on the current device are refused before any launch. No test here has a GPU: the
operands are stand-ins that know their place, and the library's functions are replaced by one that records its calls."""
import types

import pytest

torch = pytest.importorskip("torch")
import zero_gradient_reduction_gb300 as zr  # noqa: E402


class Tensor:
    """What the binding asks of a contiguous matrix or vector on a device."""

    def __init__(self, shape, dtype=torch.float32, device=0):
        self.shape, self.dtype, self._device = tuple(shape), dtype, device

    def get_device(self):
        return self._device

    @property
    def is_cuda(self):
        return self._device >= 0

    def stride(self):
        return (self.shape[1], 1)

    def element_size(self):
        return self.dtype.itemsize

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(zr, "_fns", {
        "stream": lambda device: 0, "device": lambda: 0,
        **{name: (lambda *a: made.append(a) or 0) for name in ("zr_mx4_quantize", "zr_mx4_dequantize", "zr_mx4_matmul",
                                                               "zr_mx4_linear", "zr_distill_topk")}})
    monkeypatch.setattr(zr, "_types", {torch.float16: zr.F16, torch.bfloat16: zr.BF16, torch.float32: zr.F32})
    return made


def mx4(rows, cols, device=0):
    return zr.Mx4(rows, cols, data=Tensor((zr.mx4_bytes(rows, cols),), torch.uint8, device))


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    from zero_gradient_reduction_gb300 import build as zbuild
    zbuild.build()


def operands(call):
    """(function, operands by name): each operand is made on the device that it is given."""
    if call == "quantize":
        return zr.mx4_quantize, dict(x=lambda d: Tensor((4, 64), device=d), q=lambda d: mx4(4, 64, d), q_t=lambda d: mx4(64, 4, d),
                                     rand=lambda d: Tensor((4, 64), torch.uint8, d))
    if call == "dequantize":
        return zr.mx4_dequantize, dict(q=lambda d: mx4(4, 64, d), out=lambda d: Tensor((4, 64), device=d))
    if call == "matmul":
        return zr.mx4_matmul, dict(a=lambda d: mx4(4, 64, d), b=lambda d: mx4(8, 64, d), out=lambda d: Tensor((4, 8), device=d))
    if call == "linear":
        return zr.mx4_linear, dict(x=lambda d: Tensor((4, 64), device=d), w=lambda d: mx4(8, 64, d),
                                   out=lambda d: Tensor((4, 8), device=d), xq=lambda d: mx4(4, 64, d))
    return zr.distill_topk, dict(logits=lambda d: Tensor((4, 50), device=d), ids=lambda d: Tensor((4, 3), torch.int32, d),
                                 teacher=lambda d: Tensor((4, 3), device=d), loss=lambda d: Tensor((4,), device=d),
                                 grad=lambda d: Tensor((4, 50), device=d), weight=lambda d: Tensor((4,), device=d),
                                 plan=lambda d: types.SimpleNamespace(handle=1, device=d))


CALLS = ["quantize", "dequantize", "matmul", "linear", "distill"]


@pytest.mark.parametrize("call", CALLS)
def test_together_on_the_current_device(calls, call):
    fn, makers = operands(call)
    fn(**{k: make(0) for k, make in makers.items()})
    assert len(calls) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in operands(c)[1]])
def test_one_operand_elsewhere(calls, call, name):
    fn, makers = operands(call)
    with pytest.raises(zr.ZrError) as e:
        fn(**{k: make(1 if k == name else 0) for k, make in makers.items()})
    assert e.value.status == 1 and "device" in str(e.value) and not calls


@pytest.mark.parametrize("call", CALLS)
def test_all_operands_on_a_device_that_is_not_current(calls, call):
    fn, makers = operands(call)
    with pytest.raises(zr.ZrError) as e:
        fn(**{k: make(1) for k, make in makers.items()})
    assert e.value.status == 1 and not calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(calls, call):
    fn, makers = operands(call)
    fn(**{k: make(0) for k, make in makers.items()}, stream=types.SimpleNamespace(cuda_stream=64, device_index=0))
    assert calls.pop()[-1] == 64
    with pytest.raises(zr.ZrError):
        fn(**{k: make(0) for k, make in makers.items()}, stream=types.SimpleNamespace(cuda_stream=64, device_index=1))
    assert not calls


def test_a_matrix_in_host_memory():
    """Made by the constructor itself, too: its address would go to a kernel."""
    with pytest.raises(zr.ZrError):
        zr.Mx4(4, 64, device="cpu")
    with pytest.raises(zr.ZrError):
        mx4(4, 64, device=-1)


def test_no_loss(calls):
    fn, makers = operands("distill")
    with pytest.raises(zr.ZrError) as e:
        fn(**{**{k: make(0) for k, make in makers.items()}, "loss": None})
    assert e.value.status == 1 and not calls
