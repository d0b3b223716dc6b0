"""A few tokens at the end of their buffer: rows of every length past a 16-byte word, with what is no number behind the last."""
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr
from test_mx4_gpu import BF16, F16, F32, check, matrix, on_host, quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    zr.mx4_status()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M", [1, 3, 16])
@pytest.mark.parametrize("K", [1, 7, 8, 9, 15, 17, 31, 257, 1000, 1003, 2049])
def test_last_tokens(M, K, dtype):
    x = matrix(M, K, dtype, seed=M + K)
    room = torch.full((M * K + 16,), float("nan"), dtype=dtype, device="cuda")
    room[:M * K] = x.flatten()
    w, wv = quantised(130, K, 8)
    out = torch.empty(M, 130, device="cuda")
    zr.mx4_linear(room[:M * K].view(M, K), w, out)
    check(out, ref.values(*ref.quantise(on_host(x)), K), wv)
