"""Column sums of many rows, whatever the rows' stride: sums do not lose with the number of rows.

Eight rows' values are added in three steps of fp32, which may each cost 2^-24 of them, their sums in two words, of which
the second's own roundings are 2^-48 and do not count even 10^5 times; the result is rounded once: under 5 times 2^-24 of
the sum of the magnitudes."""
import numpy as np
import pytest
import torch

import zero_gradient_reduction_gb300 as zr

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("M,N", [(8192, 2048), (70_001, 9605), (70_001, 512), (1003, 40_001), (100_003, 7), (64, 300), (9, 9)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_sums_of_one_sign(M, N, dtype):
    for ld in (N, N + 1, (N + 15) // 8 * 8):
        x = torch.empty(M, ld, dtype=dtype, device="cuda")
        x.uniform_(1.0, 1.25)
        got = torch.empty(N, device="cuda")
        zr.column_sums(x[:, :N], got)
        want = torch.zeros(N, dtype=torch.float64, device="cuda")
        for a in range(0, M, 4096):
            want += x[a:a + 4096, :N].double().sum(0)
        assert bool(((got.double() - want).abs() <= 5 * EPS * want).all()), float(((got.double() - want).abs() / want).max() / EPS)


@pytest.mark.parametrize("ld", [2048, 2051])
def test_sums_of_both_signs(ld):
    """In the root mean square no more than rounding the sums once, and the eight rows': 4e-8 of the sums'."""
    x = torch.randn(8192, ld, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)[:, :2048]
    got = torch.empty(2048, device="cuda")
    zr.column_sums(x, got)
    want = x.double().sum(0)
    assert float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt()) < 4e-8
    assert bool(((got.double() - want).abs() <= 5 * EPS * x.double().abs().sum(0)).all())


@pytest.mark.parametrize("ld", [64, 67])
def test_infinite_sums(ld):
    """An infinity stays one, two of both signs are no number, and sums past the type's largest value are infinite."""
    x = torch.ones(700, ld, device="cuda")[:, :64]
    x[500, 3], x[2, 4], x[699, 4], x[0, 5], x[1, 5] = INF, -INF, -INF, INF, -INF
    x[:, 6] = 3e38
    x[300, 7] = float("nan")
    got = torch.empty(64, device="cuda")
    zr.column_sums(x, got)
    got = got.cpu().numpy()
    assert got[3] == INF and got[4] == -INF and np.isnan(got[5]) and got[6] == INF and np.isnan(got[7]) and (got[8:] == 700).all()
