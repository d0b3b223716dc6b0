"""Values at the ends of the types, and scales far apart: 16-bit matrices through the quantiser and through the tokens'
own, and products whose blocks lie many powers of two apart."""
import numpy as np
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr
from test_mx4_gpu import BF16, F16, F32, on_host, same

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


def ends(dtype, cols=96):
    """Rows of a 16-bit type with its subnormals, its largest values, zeros of both signs, ties, and what is no number, in
    even and odd columns (the lower and the upper half of a word)."""
    tiny = 2.0 ** (-24 if dtype == F16 else -133)
    top = torch.finfo(dtype).max
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(24, cols, dtype=torch.float64)
    x[0, :4] = torch.tensor([tiny, -tiny, 0.0, -0.0])
    x[1, :4] = torch.tensor([7 * tiny, 5 * tiny, 3 * tiny, tiny])
    x[2, :3] = torch.tensor([top, -top / 2, top / 64])
    x[3, :4] = torch.tensor([torch.finfo(dtype).tiny, tiny, -torch.finfo(dtype).tiny, 2 * tiny])
    x[4, 2], x[4, 3] = 1.0, inf
    x[5, 2], x[5, 3] = inf, 1.0
    x[6, 40], x[6, 41] = nan, 2.0
    x[7, 40], x[7, 41] = 2.0, nan
    x[8, 1], x[9, 94] = -inf, -inf
    x[10, :8] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25])
    x[11, :8] = -torch.tensor([4.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25])
    x[12] = torch.linspace(-8, 8, cols)
    x[13] = torch.linspace(-1, 1, cols) * 2.0 ** (-12 if dtype == F16 else -124)
    x[14] = torch.linspace(1, 7, cols) * tiny
    x[15, ::2], x[16, 1::2] = top, tiny
    x[17, 5], x[17, 6], x[17, 70] = inf, nan, 1.0
    x[18] = -0.0
    x = x.to(dtype)
    x.view(torch.int16)[19, 9] = -1  # NaN with its sign and all bits set
    x.view(torch.int16)[20, 8] = 0x7C01 if dtype == F16 else 0x7F81  # a signalling one
    return x


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("chance", [False, True])
def test_sixteen_bit_ends_of_the_range(dtype, chance):
    x = ends(dtype)
    rows, cols = x.shape
    rand = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, generator=torch.Generator().manual_seed(4))
    q, qt = zr.Mx4(rows, cols), zr.Mx4(cols, rows)
    zr.mx4_quantize(x.cuda(), q, qt, rand=rand.cuda() if chance else None)
    h, r = x.double().numpy(), rand.numpy() if chance else None
    same(q, ref.quantise(h, r), cols)
    same(qt, ref.quantise(h.T, None if r is None else r.T), rows)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("M,buffer", [(1, False), (7, False), (16, True), (24, True)])
def test_tokens_at_the_ends_of_the_range(dtype, M, buffer):
    """Each output is one quantised token value times 1 (a weight matrix with a single 1 in each row), so it is that value;
    under 2^-126 a product may be flushed to zero. A token with a value that is no number has no finite output."""
    x = ends(BF16 if dtype == F32 else dtype).to(dtype)
    x = torch.cat([x[19 - M // 2:], x])[:M] if M < 24 else x
    K = x.shape[1]
    w = zr.Mx4(K, K)
    zr.mx4_quantize(torch.eye(K, device="cuda"), w)
    out = torch.empty(M, K, device="cuda")
    zr.mx4_linear(x.cuda(), w, out, xq=zr.Mx4(M, K) if buffer else None)
    v = ref.values(*ref.quantise(x.double().numpy()), K)
    bad = np.isnan(v).any(1)
    got = on_host(out)
    assert np.isnan(got[bad]).all()
    assert (np.abs(got[~bad] - v[~bad]) <= np.where(np.abs(v[~bad]) < 2.0 ** -126, 2.0 ** -126, 0.0)).all()


def blocks(rows, cols, exponents, seed):
    """Normal values with a power of two of their own for each block of 32: quantised, and what that stands for."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    x = (x.clamp(-3, 3) * torch.exp2(exponents.double()).repeat_interleave(32, 1)[:, :cols]).float().cuda()
    q = zr.Mx4(rows, cols)
    zr.mx4_quantize(x, q)
    return q, ref.values(*ref.quantise(on_host(x)), cols)


def check_wide(out, a, b):
    """The exact product, and what sums in fp32 may cost: the 32 products of a block add exactly (multiples of 1/4 under
    2^11, times a power of two), each of the K/32 sums of blocks that follow costs at most a truncated unit, 2^-23, of
    the sum of magnitudes, or what lies under 2^-126 where that is flushed; one rounding to the type."""
    y = a @ b.T
    terms = a.shape[1] // 32 + 2
    bound = np.abs(a) @ np.abs(b).T * terms * 2.0 ** -23 + terms * 2.0 ** -126 + ref.rounding(out.dtype, y) * (1 + 2.0 ** -10)
    d = np.abs(on_host(out) - y)
    assert (d <= bound).all(), (d / bound).max()


FORMS = [(2, 200, 1000), (16, 300, 2048), (130, 300, 1000), (64, 500, 8192), (2304, 2304, 2048)]  # few tokens, tiles, shared K, pairs


@pytest.mark.parametrize("M,N,K", FORMS)
def test_products_of_blocks_far_apart(M, N, K):
    """A row's blocks, and so the terms of its sums, lie up to 2^80 apart."""
    g = torch.Generator().manual_seed(M)
    nb = -(-K // 32)
    (a, av), (b, bv) = (blocks(r, K, torch.randint(-20, 21, (r, nb), generator=g), s) for r, s in ((M, 1), (N, 2)))
    out = torch.empty(M, N, device="cuda")
    zr.mx4_matmul(a, b, out)
    check_wide(out, av, bv)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_products_of_a_huge_and_a_tiny_block(M, N, K):
    """Scale bytes from 0 to 252 on one side against their inverses on the other: every product of blocks is near 1."""
    nb = -(-K // 32)
    e = torch.linspace(-126, 125, nb).round()
    e = e[torch.randperm(nb, generator=torch.Generator().manual_seed(5))]
    (a, av), (b, bv) = blocks(M, K, e.expand(M, nb), 1), blocks(N, K, (-e).expand(N, nb), 2)
    scales = ref.quantise(av)[1]
    assert scales.min() == 0 and scales.max() >= 251
    out = torch.empty(M, N, device="cuda")
    zr.mx4_matmul(a, b, out)
    check_wide(out, av, bv)
    if M <= zr.MX4_FEW:
        x = torch.from_numpy(av).float().cuda()  # quantising what is quantised changes nothing
        zr.mx4_linear(x, b, out)
        check_wide(out, ref.values(*ref.quantise(on_host(x)), K), bv)


@pytest.mark.parametrize("M,N,K", FORMS)
def test_products_past_the_range_are_infinite(M, N, K):
    """Past fp32, and in fp16 past 65504: infinite with the sum's sign (all terms of a row have one), never the largest value."""
    sign = torch.where(torch.arange(M) % 2 == 0, 1.0, -1.0)[:, None]
    for ea, eb, dtype in ((90, 60, F32), (90, 60, BF16), (10, 12, F16)):
        a, b = zr.Mx4(M, K), zr.Mx4(N, K)
        zr.mx4_quantize((sign * 2.0 ** ea).expand(M, K).contiguous().cuda(), a)
        zr.mx4_quantize(torch.full((N, K), 2.0 ** eb, device="cuda"), b)
        out = torch.empty(M, N, dtype=dtype, device="cuda")
        zr.mx4_matmul(a, b, out)
        assert torch.equal(out.float(), (sign * float("inf")).expand(M, N).cuda())
