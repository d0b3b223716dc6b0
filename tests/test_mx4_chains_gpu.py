"""Layers one behind the other, each beginning while the one before it ends: a residual that grows in place, an
activation's derivative in place with the bias's gradient taken from it, and a stored h read by the next launch, with the
bytes that the same calls give when each is waited for."""
import pytest
import torch

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


def mx4(rows, cols, g):
    q = zr.Mx4(rows, cols)
    zr.mx4_quantize(torch.randn(rows, cols, generator=g, device="cuda") / cols ** 0.5, q)
    return q


# pairs of blocks, blocks alone, parts of K; whole words and rows on no boundary
SHAPES = [(4096, 4096, 512, 0), (777, 520, 300, 0), (64, 1024, 4096, 0), (300, 513, 256, 2), (8, 2048, 2048, 0)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,N,K,more", SHAPES)
def test_chains(M, N, K, more, dtype):
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b, bias = mx4(M, K, g), mx4(N, K, g), torch.randn(N, generator=g, device="cuda")
    first = torch.randn(M, N + more, generator=g, device="cuda").to(dtype)

    def chain(wait):
        y, h, z = first.clone()[:, :N], torch.empty(M, N + more, dtype=dtype, device="cuda")[:, :N], torch.empty(M, N, dtype=dtype, device="cuda")
        db = torch.empty(8, N, device="cuda")
        torch.cuda.synchronize()
        for i in range(8):
            zr.mx4_matmul(a, b, y, bias=bias, residual=y)  # y grows in place
            wait()
            zr.mx4_matmul(a, b, z, activation="gelu", residual=y, pre=h)
            wait()
            zr.mx4_matmul(a, b, h, gradient_of="silu", pre=h)
            wait()
            zr.column_sums(h, db[i])
            wait()
            zr.mx4_matmul(a, b, y, residual=z)
            wait()
        torch.cuda.synchronize()
        return y.clone(), h.clone(), z, db

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(x, w) for x, w in zip(chain(lambda: None), want))
    zr.mx4_status()
