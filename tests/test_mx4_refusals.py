"""Arguments that the 4-bit and distillation calls refuse, before any CUDA call and so without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    from zero_gradient_reduction_gb300 import build as zbuild
    zbuild.build()
    import zero_gradient_reduction_gb300 as z
    return z.lib()


def refused(L, status, word):
    assert status == 1, status
    assert word in L.zr_last_error().decode(), L.zr_last_error()


def test_bytes(L):
    assert L.zr_mx4_bytes(0, 5) == 0 and L.zr_mx4_bytes(5, 0) == 0 and L.zr_mx4_bytes(-1, 5) == -1
    assert L.zr_mx4_bytes(1, 1) == 17408 and L.zr_mx4_bytes(129, 257) == 4 * 17408
    assert L.zr_mx4_bytes(1 << 20, 1 << 20) == (1 << 13) * (1 << 12) * 17408  # past 32 bits


def test_quantize(L):
    q = L.zr_mx4_quantize
    refused(L, q(16, 5, 4, 32, 32, None, 0, 16, None, None), "dtype")
    refused(L, q(16, 2, -1, 32, 32, None, 0, 16, None, None), "negative")
    refused(L, q(16, 2, 4, 32, 31, None, 0, 16, None, None), "stride")
    refused(L, q(16, 2, 4, 32, 32, 16, 31, 16, None, None), "stride")
    refused(L, q(16, 2, 4, 32, 32, None, 0, None, None, None), "neither")
    refused(L, q(None, 2, 4, 32, 32, None, 0, 16, None, None), "null")
    for bad in ((24, None, 16, None), (16, 24, 16, None), (16, None, 24, None), (16, None, 16, 24)):
        refused(L, q(bad[0], 2, 4, 32, 32, bad[1], 32, bad[2], bad[3], None), "aligned")
    assert q(None, 2, 0, 32, 32, None, 0, 16, None, None) == 0


def test_dequantize(L):
    d = L.zr_mx4_dequantize
    refused(L, d(16, 4, 32, 16, 3, 32, None), "dtype")
    refused(L, d(16, 4, -2, 16, 2, 32, None), "negative")
    refused(L, d(16, 4, 32, 16, 2, 8, None), "stride")
    refused(L, d(None, 4, 32, 16, 2, 32, None), "null")
    refused(L, d(16, 4, 32, 18, 2, 32, None), "aligned")


def test_products(L):
    m, x = L.zr_mx4_matmul, L.zr_mx4_linear
    refused(L, m(16, 4, 16, 8, 32, 16, 9, 8, None), "dtype")
    refused(L, m(16, 4, 16, -8, 32, 16, 2, 8, None), "negative")
    refused(L, m(16, 4, 16, 8, 32, 16, 2, 7, None), "stride")
    refused(L, m(16, 4, None, 8, 32, 16, 2, 8, None), "null")
    refused(L, m(16, 4, 16, 8, 32, None, 2, 8, None), "null")
    refused(L, m(8, 4, 16, 8, 32, 16, 2, 8, None), "aligned")
    refused(L, x(16, 3, 4, 32, 16, 8, 32, 16, 2, 8, None, None), "dtype")
    refused(L, x(16, 2, 4, 31, 16, 8, 32, 16, 2, 8, None, None), "stride")
    refused(L, x(16, 2, 4, 32, 16, 8, 32, 16, 2, 7, None, None), "stride")
    refused(L, x(16, 2, 4, 32, None, 8, 32, 16, 2, 8, None, None), "null")
    refused(L, x(16, 2, 4, 32, 16, 8, 32, 16, 2, 8, 8, None), "aligned")
    assert m(None, 0, None, 8, 32, None, 2, 8, None) == 0


def test_distill(L):
    def call(**k):
        a = dict(z=16, dt=2, T=4, V=100, ldz=100, ids=16, ids64=0, teacher=16, tdt=2, K=3, ldk=3, weight=None, tau=1.0,
                 scale=1.0, plan=None, loss=16, grad=1 << 20, ldg=100)
        a.update(k)
        return L.zr_distill_topk(a["z"], a["dt"], a["T"], a["V"], a["ldz"], a["ids"], a["ids64"], a["teacher"], a["tdt"],
                                 a["K"], a["ldk"], a["weight"], a["tau"], a["scale"], a["plan"], a["loss"], a["grad"], a["ldg"], None)

    refused(L, call(dt=7), "dtype")
    refused(L, call(tdt=-1), "dtype")
    refused(L, call(V=0, ldz=0), "V")
    refused(L, call(K=0), "K=")
    refused(L, call(K=1025, ldk=1025), "K=")
    for k in ("ldz", "ldg"):
        refused(L, call(**{k: 99}), "stride")
    refused(L, call(ldk=2), "stride")
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        refused(L, call(tau=tau), "temperature")
    for s in (float("nan"), float("inf")):
        refused(L, call(scale=s), "grad_scale")
    for k in ("z", "ids", "teacher", "loss"):
        refused(L, call(**{k: None}), "null")
        refused(L, call(**{k: 24}), "aligned")
    refused(L, call(grad=32), "overlaps")
    refused(L, call(grad=16, ldg=104), "overlaps")
    assert call(T=0) == 0


def test_binding_refuses_what_the_library_cannot_see(L):
    torch = pytest.importorskip("torch")
    import zero_gradient_reduction_gb300 as zr
    with pytest.raises(zr.ZrError):
        zr.Mx4(-1, 4, data=torch.empty(0, dtype=torch.uint8))
    with pytest.raises(zr.ZrError):
        zr.Mx4(4, 4, data=torch.empty(17408, dtype=torch.uint8))  # not device memory
    with pytest.raises(zr.ZrError):
        zr.mx4_quantize(torch.zeros(4, 4))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
