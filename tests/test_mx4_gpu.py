"""Microscaled 4-bit matrices on the GPU against the format's definition in 64 bits: quantisation and its layout,
the products, and where they can go wrong."""
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
    yield
    zr.mx4_status()  # no product gave up a wait


def matrix(rows, cols, dtype, seed=0, ld=None, wide=True):
    """Values over many powers of two, some blocks zero, some values right between two neighbours."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    if wide:
        x *= torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
        grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.0])
        hit = torch.rand(rows, cols, generator=g) < 0.3
        x = torch.where(hit, grid[torch.randint(0, 9, (rows, cols), generator=g)] * torch.sign(x), x)
        x[torch.rand(rows, generator=g) < 0.1] = 0
    x = x.to(dtype)
    if ld is None:
        return x.cuda()
    room = torch.full((rows, ld), float("nan"), dtype=dtype, device="cuda")
    room[:, :cols] = x.cuda()
    return room[:, :cols]


def on_host(t):
    return t.detach().double().cpu().numpy()


def same(got, want, cols):
    """The bytes of a 4-bit matrix against codes and scale bytes."""
    code, byte = want
    np.testing.assert_array_equal(got.data.cpu().numpy(), ref.layout(code, byte))


SIZES = [(1, 1), (1, 31), (2, 32), (3, 33), (1, 300), (128, 256), (129, 257), (255, 130), (300, 1000), (40, 2049)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("chance", [False, True])
def test_quantise_both_ways(rows, cols, dtype, chance):
    x = matrix(rows, cols, dtype, seed=rows + cols)
    rand = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, generator=torch.Generator().manual_seed(1)).cuda() if chance else None
    q, qt = zr.Mx4(rows, cols), zr.Mx4(cols, rows)
    q.data.fill_(0xEE), qt.data.fill_(0xEE)
    zr.mx4_quantize(x, q, qt, rand=rand)
    h, r = on_host(x), None if rand is None else rand.cpu().numpy()
    same(q, ref.quantise(h, r), cols)
    same(qt, ref.quantise(h.T, None if r is None else r.T), rows)
    for both in (q, None), (None, qt):  # one of the two alone gives the same bytes
        one = zr.Mx4(rows, cols) if both[0] else None
        two = zr.Mx4(cols, rows) if both[1] else None
        zr.mx4_quantize(x, one, two, rand=rand)
        assert torch.equal((one or two).data, (both[0] or both[1]).data)


@pytest.mark.parametrize("dtype,ld", [(F32, 301), (F32, 304), (F16, 301), (F16, 302), (BF16, 303), (BF16, 308), (BF16, 312)])
def test_quantise_row_strides(dtype, ld):
    x = matrix(77, 300, dtype, seed=ld, ld=ld)
    q, qt = zr.Mx4(77, 300), zr.Mx4(300, 77)
    zr.mx4_quantize(x, q, qt)
    same(q, ref.quantise(on_host(x)), 300)
    same(qt, ref.quantise(on_host(x).T), 77)


@pytest.mark.parametrize("chance", [False, True])
def test_quantise_ends_of_the_range(chance):
    """Subnormals, the largest values, one bit over and under 6 of the scale, signed zeros, and values that are not finite."""
    x = torch.zeros(12, 64)
    x[0, :4] = torch.tensor([1e-45, -1e-45, 0.0, -0.0])
    x[1, :4] = torch.tensor([2.0 ** -127, -(2.0 ** -128), 2.0 ** -126, 3e-39])
    x[2, :3] = torch.tensor([3.4028235e38, -1e38, 1e30])
    x[3, :3] = torch.tensor([6.0, np.nextafter(np.float32(6), np.float32(7)), 0.1])
    x[4, :3] = torch.tensor([6.0, 0.25, 0.25000003])
    x[5, 3] = float("inf")
    x[6, 40] = float("nan")
    x[7, :2] = torch.tensor([float("-inf"), 3.0])
    x[8, :3] = torch.tensor([7.9999995, 4.9999995, 5.0])
    x[9] = torch.linspace(-8, 8, 64)
    x[10] = torch.linspace(-1, 1, 64) * 2.0 ** -125
    x[11, ::2] = 2.0 ** -120
    rand = torch.randint(0, 256, x.shape, dtype=torch.uint8, generator=torch.Generator().manual_seed(3))
    q, qt = zr.Mx4(12, 64), zr.Mx4(64, 12)
    zr.mx4_quantize(x.cuda(), q, qt, rand=rand.cuda() if chance else None)
    r = rand.numpy() if chance else None
    code, byte = ref.quantise(x.numpy(), r)
    same(q, (code, byte), 64)
    same(qt, ref.quantise(x.numpy().T, r.T if chance else None), 12)
    out = torch.empty(12, 64, device="cuda")
    zr.mx4_dequantize(q, out)
    want = torch.from_numpy(ref.values(code, byte, 64)).float()  # rounded up by chance the largest value is 2^128: infinite in fp32
    np.testing.assert_array_equal(out.cpu().numpy(), want.numpy())


def test_rounding_by_chance_keeps_the_mean():
    """Over all 256 random bytes the mean is the value, to half of the step's 1/256 that the bytes resolve."""
    x = matrix(16, 256, F32, seed=5, wide=False)
    total = torch.zeros(16, 256, dtype=torch.float64, device="cuda")
    q, out = zr.Mx4(16, 256), torch.empty(16, 256, device="cuda")
    for r in range(256):
        zr.mx4_quantize(x, q, rand=torch.full((16, 256), r, dtype=torch.uint8, device="cuda"))
        zr.mx4_dequantize(q, out)
        total += out.double()
    step = x.view(16, 8, 32).abs().amax(2, keepdim=True).expand(16, 8, 32).reshape(16, 256)  # the largest spacing is under the largest magnitude
    assert bool(((total / 256 - x.double()).abs() <= step.double() / 512).all())


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 33), (130, 300), (257, 1001)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_dequantise(rows, cols, dtype):
    x = matrix(rows, cols, F32, seed=9)
    q = zr.Mx4(rows, cols)
    zr.mx4_quantize(x, q)
    want = torch.from_numpy(ref.values(*ref.quantise(on_host(x)), cols)).to(dtype)
    for ld in (cols, cols + 3, (cols + 15) // 8 * 8):
        room = torch.full((rows, ld), 7.0, dtype=dtype, device="cuda")
        zr.mx4_dequantize(q, room[:, :cols])
        assert torch.equal(room[:, :cols].cpu(), want)
        assert bool((room[:, cols:] == 7.0).all())


def product(a, b, dtype):
    """What A B^T may be: the exact product, and how far fp32 sums in any order and one rounding to the type may lie
    from it. A sum of n terms costs at most (n - 1) units of 2^-23 (truncated additions) of the sum of magnitudes; 32
    products of a block are exact before it, as multiples of 1/4 under 2^11."""
    y = a @ b.T
    magnitude = np.abs(a) @ np.abs(b).T
    return y, magnitude * (a.shape[1] // 32 + 2) * 2.0 ** -23 + ref.rounding(dtype, y) * (1 + 2.0 ** -10)


def check(out, a, b):
    y, bound = product(a, b, out.dtype)
    d = np.abs(on_host(out) - y)
    assert (d <= bound).all(), (d - bound).max()


def quantised(rows, cols, seed):
    x = matrix(rows, cols, F32, seed=seed, wide=False) * 3
    q = zr.Mx4(rows, cols)
    zr.mx4_quantize(x, q)
    return q, ref.values(*ref.quantise(on_host(x)), cols)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 7, 31), (128, 128, 256), (127, 129, 255), (129, 257, 257), (130, 64, 1000), (300, 515, 768), (16, 1000, 513)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_matmul(M, N, K, dtype):
    (a, av), (b, bv) = quantised(M, K, 1), quantised(N, K, 2)
    for ld in (N, N + 5, (N + 15) // 8 * 8):
        room = torch.full((M, ld), 7.0, dtype=dtype, device="cuda")
        zr.mx4_matmul(a, b, room[:, :N])
        check(room[:, :N], av, bv)
        assert bool((room[:, N:] == 7.0).all())


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_matmul_more_tiles_than_multiprocessors(dtype):
    """Sizes past both tile shapes' thresholds: blocks that take several tiles, the last ones ragged; a last round that
    is taken in halves (9 x 9 tiles of 256 on 76 pairs), with a last column that is whole or a row short."""
    for M, N, K in ((2600, 3000, 512), (1100, 2699, 300), (2945, 2818, 256), (2300, 2304, 700), (2180, 2296, 512), (2304, 2181, 300)):
        (a, av), (b, bv) = quantised(M, K, 3), quantised(N, K, 4)
        for ld in (N, (N + 15) // 8 * 8):
            room = torch.full((M, ld), 7.0, dtype=dtype, device="cuda")
            zr.mx4_matmul(a, b, room[:, :N])
            check(room[:, :N], av, bv)
            assert bool((room[:, N:] == 7.0).all())


def test_matmul_is_repeatable():
    (a, _), (b, _) = quantised(700, 2000, 5), quantised(1500, 2000, 6)
    one, two = torch.empty(700, 1500, device="cuda"), torch.empty(700, 1500, device="cuda")
    zr.mx4_matmul(a, b, one)
    zr.mx4_matmul(a, b, two)
    assert torch.equal(one, two)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 13, 16, 17, 40])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 256), (300, 1000), (2309, 777), (640, 4096), (20000, 512)])
def test_linear(M, N, K):
    dtype = [F32, F16, BF16][M % 3]
    x = matrix(M, K, dtype, seed=M + N, ld=[None, K + 1, (K + 23) // 8 * 8][N % 3])
    w, wv = quantised(N, K, 8)
    xv = ref.values(*ref.quantise(on_host(x)), K)
    for out_dtype in (F32, BF16):
        room = torch.full((M, N + 3), 7.0, dtype=out_dtype, device="cuda")
        zr.mx4_linear(x, w, room[:, :N], xq=zr.Mx4(M, K) if M > zr.MX4_FEW else None)
        check(room[:, :N], xv, wv)
        assert bool((room[:, N:] == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(3, 256, 20000), (2, 200, 70000), (16, 100, 120000)])
def test_linear_long_rows(M, N, K):
    """K that fills a block's shared memory, or that only a cluster or the buffered form holds."""
    x = matrix(M, K, BF16, seed=K)
    w, wv = quantised(N, K, 8)
    out = torch.empty(M, N, device="cuda")
    zr.mx4_linear(x, w, out, xq=zr.Mx4(M, K))
    check(out, ref.values(*ref.quantise(on_host(x)), K), wv)


@pytest.mark.parametrize("M", [4, 200])
def test_not_a_number_stays_in_its_rows(M):
    """An infinity in one token makes that token's outputs NaN and no other's; one in a weight row that column."""
    x = matrix(M, 600, F32, seed=2, wide=False)
    x[1, 599] = float("inf")
    wx = matrix(300, 600, F32, seed=3, wide=False)
    wx[7, 0] = float("nan")
    w = zr.Mx4(300, 600)
    zr.mx4_quantize(wx, w)
    out = torch.empty(M, 300, device="cuda")
    zr.mx4_linear(x, w, out, xq=zr.Mx4(M, 600))
    nan = torch.isnan(out).cpu()
    want = torch.zeros(M, 300, dtype=torch.bool)
    want[1], want[:, 7] = True, True
    assert torch.equal(nan, want)
    x[1, 599] = 0
    clean = torch.empty(M, 300, device="cuda")
    zr.mx4_linear(x, w, clean, xq=zr.Mx4(M, 600))
    keep = ~want
    assert torch.equal(out.cpu()[keep], clean.cpu()[keep])


def test_what_does_not_fit_is_refused():
    """Shapes, types, places and strides that the binding sees, and the library's own refusals through it."""
    x, q = torch.zeros(8, 64, device="cuda"), zr.Mx4(8, 64)
    out = torch.empty(8, 8, device="cuda")
    for call in (lambda: zr.mx4_quantize(x, zr.Mx4(8, 65)), lambda: zr.mx4_quantize(x, None, zr.Mx4(8, 64)),
                 lambda: zr.mx4_quantize(x), lambda: zr.mx4_quantize(x.t(), zr.Mx4(64, 8)),
                 lambda: zr.mx4_quantize(x.double(), q), lambda: zr.mx4_quantize(x[:, 1:], zr.Mx4(8, 63)),
                 lambda: zr.mx4_quantize(x, q, rand=torch.zeros(8, 63, dtype=torch.uint8, device="cuda")),
                 lambda: zr.mx4_quantize(x, q, rand=x), lambda: zr.mx4_quantize(x[0], q), lambda: zr.mx4_quantize(x.expand(8, 64)[:1].expand(8, 64), q),
                 lambda: zr.mx4_dequantize(q, out), lambda: zr.mx4_matmul(q, zr.Mx4(8, 32), out),
                 lambda: zr.mx4_matmul(q, zr.Mx4(9, 64), out), lambda: zr.mx4_linear(x, zr.Mx4(9, 64), out),
                 lambda: zr.mx4_linear(torch.zeros(17, 64, device="cuda"), q, torch.empty(17, 8, device="cuda")),
                 lambda: zr.mx4_linear(x, q, out, xq=zr.Mx4(8, 65)), lambda: zr.Mx4(8, 64, data=torch.empty(17407, dtype=torch.uint8, device="cuda")),
                 lambda: zr.Mx4(8, 64, data=torch.empty(17408, device="cuda")), lambda: zr.Mx4(8, -1)):
        with pytest.raises(zr.ZrError) as e:
            call()
        assert e.value.status == 1


def test_empty_sizes():
    out = torch.full((4, 6), 7.0, device="cuda")
    zr.mx4_matmul(zr.Mx4(4, 0), zr.Mx4(6, 0), out)
    assert bool((out == 0).all())
    zr.mx4_matmul(zr.Mx4(0, 32), zr.Mx4(6, 32), torch.empty(0, 6, device="cuda"))
    zr.mx4_matmul(zr.Mx4(4, 32), zr.Mx4(0, 32), torch.empty(4, 0, device="cuda"))
    zr.mx4_quantize(torch.empty(0, 40, device="cuda"), zr.Mx4(0, 40), zr.Mx4(40, 0))
    zr.mx4_dequantize(zr.Mx4(3, 0), torch.empty(3, 0, device="cuda"))
    zr.mx4_linear(torch.empty(3, 0, device="cuda"), zr.Mx4(5, 0), out[:3, :5])
    assert bool((out[:3, :5] == 0).all())


def test_bytes_outside_are_untouched():
    """Outputs between guard bands: a 4-bit matrix's bytes, and a product's rows."""
    for rows, cols in ((1, 1), (129, 300)):
        need = zr.mx4_bytes(rows, cols)
        raw = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        zr.mx4_quantize(matrix(rows, cols, BF16), zr.Mx4(rows, cols, data=raw[4096:4096 + need]))
        assert bool((raw[:4096] == 0x5A).all()) and bool((raw[4096 + need:] == 0x5A).all())
    (a, _), (b, _) = quantised(130, 64, 1), quantised(131, 64, 2)
    raw = torch.full((130 * 131 + 2048,), 7.0, device="cuda")
    zr.mx4_matmul(a, b, raw[1024:1024 + 130 * 131].view(130, 131))
    assert bool((raw[:1024] == 7).all()) and bool((raw[1024 + 130 * 131:] == 7).all())


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 values, whose 4-bit forms are read and written past 2^32 bytes of fp32: rows and columns
    at both ends against the format's definition, and a product of more than 2^31 results."""
    rows, cols = 70_001, 32_000
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_()
    assert x.numel() > 1 << 31
    q, qt = zr.Mx4(rows, cols), zr.Mx4(cols, rows)
    zr.mx4_quantize(x, q, qt)
    out = torch.empty(rows, cols, dtype=BF16, device="cuda")
    zr.mx4_dequantize(q, out)
    for at in (slice(0, 2), slice(35_000, 35_002), slice(rows - 2, rows)):
        want = torch.from_numpy(ref.values(*ref.quantise(on_host(x[at])), cols)).to(BF16)
        assert torch.equal(out[at].cpu(), want)
    del out
    out_t = torch.empty(cols, rows, dtype=BF16, device="cuda")
    zr.mx4_dequantize(qt, out_t)
    for at in (slice(0, 2), slice(cols - 2, cols)):
        want = torch.from_numpy(ref.values(*ref.quantise(on_host(x[:, at]).T), rows)).to(BF16)
        assert torch.equal(out_t[at].cpu(), want)
    del out_t, x, q, qt
    (a, av), (b, bv) = quantised(rows, 96, 1), quantised(cols, 96, 2)
    y = torch.empty(rows, cols, dtype=BF16, device="cuda")
    zr.mx4_matmul(a, b, y)
    for at in (slice(0, 3), slice(rows - 3, rows)):
        check(y[at], av[at], bv)


def test_other_stream_and_graph():
    """A call on its own stream, and a captured quantise + product that follows its inputs."""
    x = matrix(40, 512, BF16, seed=1)
    w, wv = quantised(384, 512, 2)
    xq, out = zr.Mx4(40, 512), torch.empty(40, 384, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    zr.mx4_linear(x, w, out, xq=xq, stream=side)
    side.synchronize()
    check(out, ref.values(*ref.quantise(on_host(x)), 512), wv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        zr.mx4_linear(x, w, out, xq=xq, stream=side)
        zr.mx4_linear(x[:3], w, out[:3], stream=side)
    x.copy_(matrix(40, 512, BF16, seed=7))
    graph.replay()
    torch.cuda.synchronize()
    check(out, ref.values(*ref.quantise(on_host(x)), 512), wv)


def test_linear_layer_gradients():
    """The two products of a linear layer's backward against the formula, and against differences of the forward
    product: y is linear in each quantised operand, so a difference is exact up to the rounding of y."""
    T, N, K = 200, 160, 96
    x, w, dy = (matrix(r, c, F32, seed=s, wide=False) for r, c, s in ((T, K, 1), (N, K, 2), (T, N, 3)))
    xq, xt, wq, wt, gq, gt = (zr.Mx4(*s) for s in ((T, K), (K, T), (N, K), (K, N), (T, N), (N, T)))
    zr.mx4_quantize(x, xq, xt)
    zr.mx4_quantize(w, wq, wt)
    zr.mx4_quantize(dy, gq, gt)
    dx, dw = torch.empty(T, K, device="cuda"), torch.empty(N, K, device="cuda")
    zr.mx4_matmul(gq, wt, dx)
    zr.mx4_matmul(gt, xt, dw)
    h = [on_host(v) for v in (x, w, dy)]
    by_col = lambda v: ref.values(*ref.quantise(v.T), v.shape[0])  # noqa: E731
    check(dx, ref.values(*ref.quantise(h[2]), N), by_col(h[1]))
    check(dw, by_col(h[2]), by_col(h[0]))
    # f(W) = sum(dy * (x W^T)) at W + e and W - e in one element that the format holds exactly
    xv = ref.values(*ref.quantise(h[0]), K)
    probe = torch.zeros(N, K, device="cuda")
    ys = []
    for sign in (1.0, -1.0):
        probe[5, 9] = sign
        zr.mx4_quantize(probe, wq)
        y = torch.empty(T, N, device="cuda")
        zr.mx4_matmul(xq, wq, y)
        ys.append(on_host(y))
    difference = (h[2] * (ys[0] - ys[1])).sum() / 2
    formula = (h[2].T @ xv)[5, 9]
    assert abs(difference - formula) <= 2.0 ** -20 * (np.abs(h[2].T) @ np.abs(xv))[5, 9]


@pytest.mark.parametrize("kind", ["few", "few in clusters", "few, tokens quantised before", "alone", "pairs"])
def test_waits_end_and_say_so(kind):
    """Stages that expect bytes which nothing copies: every wait gives up after its two seconds, the status says so
    once, and the next product is right."""
    M, N, K = {"few": (2, 50000, 300), "few in clusters": (2, 500, 2048), "few, tokens quantised before": (16, 50000, 2048),
               "alone": (100, 300, 2048), "pairs": (2304, 2304, 2048)}[kind]
    x = matrix(M, K, BF16, seed=1, wide=False)
    w, wv = quantised(N, K, 2)
    xq, out = zr.Mx4(M, K), torch.empty(M, N, device="cuda")
    torch.cuda.synchronize()
    zr.lib().zr_mx4_stall_waits(1)
    try:
        zr.mx4_linear(x, w, out, xq=xq)
    finally:
        zr.lib().zr_mx4_stall_waits(0)
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5
    zr.mx4_status()
    zr.mx4_linear(x, w, out, xq=xq)
    check(out[:, :400], ref.values(*ref.quantise(on_host(x)), K), wv[:400])


@pytest.mark.parametrize("M,N,K", [(1100, 2699, 4100), (2300, 2304, 3900), (2304, 2181, 4096), (2180, 2296, 4096), (1024, 4096, 4096)])
def test_matmul_of_a_long_k_by_pairs(M, N, K):
    """Where K is long pairs of blocks take 256 x 256 tiles: a round that leaves pairs free, ragged last tiles, and a
    last round in halves with a last column that is whole or a row short."""
    (a, av), (b, bv) = quantised(M, K, 7), quantised(N, K, 8)
    for dtype in (F32, F16, BF16):
        for ld in (N, (N + 15) // 8 * 8):
            room = torch.full((M, ld), 7.0, dtype=dtype, device="cuda")
            zr.mx4_matmul(a, b, room[:, :N])
            check(room[:, :N], av, bv)
            assert bool((room[:, N:] == 7.0).all())


def test_waits_of_pairs_end_and_say_so():
    (a, av), (b, bv) = quantised(2304, 4096, 1), quantised(2304, 4096, 2)
    out = torch.empty(2304, 2304, device="cuda")
    torch.cuda.synchronize()
    zr.lib().zr_mx4_stall_waits(1)
    try:
        zr.mx4_matmul(a, b, out)
    finally:
        zr.lib().zr_mx4_stall_waits(0)
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5
    zr.mx4_status()
    zr.mx4_matmul(a, b, out)
    check(out[:, :400], av, bv[:400])


def test_a_chain_of_launches_reads_what_the_one_before_wrote():
    """Products and dequantisations begin while the launch before them ends: each of a chain reads its output."""
    (w, wv), x = quantised(512, 512, 3), matrix(512, 512, BF16, seed=4, wide=False)
    q, y, back = zr.Mx4(512, 512), torch.empty(512, 512, device="cuda"), torch.empty(512, 512, device="cuda")
    want = None
    for turn in range(20):
        zr.mx4_quantize(x, q)
        zr.mx4_matmul(q, w, y)
        zr.mx4_quantize(y, q)
        zr.mx4_dequantize(q, back)
        zr.mx4_matmul(q, w, y)
        got = (y.clone(), back.clone())
        if turn == 0:
            torch.cuda.synchronize()
            want = got
            first = np.zeros((512, 512))
            first[:] = ref.values(*ref.quantise(on_host(x)), 512) @ wv.T
            qv = ref.values(*ref.quantise(first.astype(np.float32).astype(np.float64)), 512)
            assert (np.abs(on_host(back) - qv) > 0).mean() < 0.01  # a rounding of fp32 sums apart
            check(y, on_host(back), wv)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("M,N,K", [(17, 300, 4100), (40, 77, 5000), (64, 2048, 8192), (129, 901, 8192), (640, 1100, 8200), (1, 5, 100_001)])
def test_matmul_of_few_tiles_and_a_long_k(M, N, K):
    """Clusters of 2, 4 and 8 blocks share K: parts of unequal length, tiles of one row and of 128, every output type."""
    (a, av), (b, bv) = quantised(M, K, 9), quantised(N, K, 10)
    for dtype in (F32, F16, BF16):
        for ld in (N, N + 3, (N + 15) // 8 * 8):
            room = torch.full((M, ld), 7.0, dtype=dtype, device="cuda")
            zr.mx4_matmul(a, b, room[:, :N])
            check(room[:, :N], av, bv)
            assert bool((room[:, N:] == 7.0).all())
            again = torch.empty_like(room)
            zr.mx4_matmul(a, b, again[:, :N])
            assert torch.equal(again[:, :N], room[:, :N])


def test_waits_of_blocks_that_share_k_end_and_say_so():
    (a, av), (b, bv) = quantised(64, 8192, 1), quantised(512, 8192, 2)
    out = torch.empty(64, 512, device="cuda")
    torch.cuda.synchronize()
    zr.lib().zr_mx4_stall_waits(1)
    try:
        zr.mx4_matmul(a, b, out)
    finally:
        zr.lib().zr_mx4_stall_waits(0)
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5
    zr.mx4_status()
    zr.mx4_matmul(a, b, out)
    check(out, av, bv)


def test_captured_behind_copies_and_other_streams():
    """Products and dequantisations as a graph's first node, behind a copy, a fill and a kernel of torch, and behind a
    join of two streams: each replay gives what the calls give one by one."""
    (a, av), (b, bv) = quantised(300, 700, 11), quantised(200, 700, 12)
    a2 = zr.Mx4(300, 700)
    out, back, moved = torch.empty(300, 200, device="cuda"), torch.empty(300, 700, device="cuda"), torch.empty(300, 200, device="cuda")
    x = matrix(300, 700, F32, seed=13, wide=False)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        zr.mx4_matmul(a, b, out)            # first
        moved.copy_(out)
        a2.data.copy_(a.data)
        zr.mx4_dequantize(a2, back)         # behind a copy
        back.add_(1.0)
        out.zero_()
        zr.mx4_matmul(a2, b, out)           # behind a fill
        out.mul_(2.0)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            zr.mx4_quantize(x, a2)
        moved.add_(out)
        here.wait_stream(side)
        zr.mx4_matmul(a2, b, out)           # behind a join

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        work()
    main.synchronize()
    want = [t.clone() for t in (out, back, moved, a2.data)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        work()
    for _ in range(3):
        for t in (out, back, moved):
            t.fill_(7.0)
        a2.data.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((out, back, moved, a2.data), want):
            assert torch.equal(got, w)
    check(out, ref.values(*ref.quantise(on_host(x)), 700), bv)
    assert np.array_equal(on_host(back), (av.astype(np.float32) + np.float32(1)).astype(np.float64))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ld", [320, 322, 324, 328, 321])
@pytest.mark.parametrize("cols", [304, 312, 308, 306, 301])
def test_quantise_row_strides_of_values_and_random_bytes(dtype, ld, cols):
    """Rows that begin on boundaries of 16, 8, 4 and fewer bytes: the values' by ld, the random bytes' by cols."""
    rows = 131
    x = matrix(rows, cols, dtype, seed=ld, ld=ld)
    rand = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, generator=torch.Generator().manual_seed(cols)).cuda()
    q, qt = zr.Mx4(rows, cols), zr.Mx4(cols, rows)
    zr.mx4_quantize(x, q, qt, rand=rand)
    h, r = on_host(x), rand.cpu().numpy()
    same(q, ref.quantise(h, r), cols)
    same(qt, ref.quantise(h.T, r.T), rows)
