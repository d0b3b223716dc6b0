"""Products of 4-bit matrices with bias, activation and residual, the products behind an activation in the backward pass, and
column sums, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import _mx4_ref as ref
import zero_gradient_reduction_gb300 as zr
from test_mx4_gpu import BF16, F16, F32, matrix, on_host, product

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)
    yield
    zr.mx4_status()


def logistic(u):
    return np.where(u >= 0, 1 / (1 + np.exp(-np.abs(u))), np.exp(-np.abs(u)) / (1 + np.exp(-np.abs(u))))


def parts(h, name):
    """(u, du/dh) of h S(u)."""
    if name == "gelu":
        c = math.sqrt(8 / math.pi)
        return c * (h + 0.044715 * h ** 3), c * (1 + 3 * 0.044715 * h ** 2)
    return h, np.ones_like(h)


def activation(h, e_h, name):
    """(value, what it may be off by) for an h that is off by e_h. The slopes lie under 1.13. An exponent of u carries up to
    eight roundings of its size, the exponential and the reciprocal two units each, the product one."""
    if name is None:
        return h, e_h
    if name == "relu":
        return np.maximum(h, 0), e_h
    u, _ = parts(h, name)
    y = h * logistic(u)
    return y, 1.13 * e_h + np.abs(y) * EPS * (8 * np.minimum(np.abs(u), 200) + 16) + 2.0 ** -120 * (1 + np.abs(h))


def derivative(h, name):
    """(value, what its arithmetic may cost): as above, of both terms."""
    if name == "relu":
        return np.where(h > 0, 1.0, 0.0), 0.0
    u, du = parts(h, name)
    first, second = logistic(u), h * logistic(u) * logistic(-u) * du
    return first + second, (first + np.abs(second)) * EPS * (10 * np.minimum(np.abs(u), 200) + 20) + 2.0 ** -100


def rounded(y, e, dtype):
    return e + (ref.rounding(dtype, np.abs(y) + e)) * (1 + 2.0 ** -10) + (2.0 ** -149 if dtype == F32 else 0)


def operand(rows, cols, seed, scale):
    x = matrix(rows, cols, F32, seed=seed, wide=False) * scale
    q = zr.Mx4(rows, cols)
    zr.mx4_quantize(x, q)
    return x, q, ref.values(*ref.quantise(on_host(x)), cols)


def expect(av, bv, bias, act, residual, dtype):
    """((out, bound), (h, bound)) of the forward form."""
    s, e = product(av, bv, F32)
    h = s if bias is None else s + on_host(bias)
    e_h = e + EPS * np.abs(h) + (0 if bias is None else EPS * e)
    y, e_y = activation(h, e_h, act)
    if residual is not None:
        y = y + on_host(residual)
        e_y = e_y + EPS * (np.abs(y) + e_y)
    return (y, rounded(y, e_y, dtype)), (h, rounded(h, e_h, dtype))


def near(got, want, bound, what):
    d = np.abs(on_host(got) - want)
    assert (d <= bound).all(), (what, float((d - bound).max()), np.argwhere(~(d <= bound))[:4])


def room_for(M, N, ld, dtype, value=7.0):
    return torch.full((M, ld), value, dtype=dtype, device="cuda")


SIZES = [(1, 1, 1), (5, 7, 31), (128, 128, 256), (129, 257, 257), (130, 64, 1000), (300, 515, 768), (64, 520, 8192), (20, 1000, 4096)]
KINDS = [(None, True, False, False), ("relu", False, True, True), ("gelu", True, False, True), ("silu", True, True, False), (None, False, True, False)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_matmul(M, N, K, dtype):
    _, a, av = operand(M, K, 1, 1.0)
    _, b, bv = operand(N, K, 2, 1.5 / math.sqrt(K))
    g = torch.Generator().manual_seed(M)
    for i, (act, has_bias, has_residual, has_pre) in enumerate(KINDS):
        ld = (N, N + 5, (N + 15) // 8 * 8)[i % 3]
        bias = torch.randn(N, generator=g).to((F32, BF16, F16)[i % 3]).cuda() if has_bias else None
        residual = torch.randn(M, ld, generator=g).to(dtype).cuda()[:, :N] if has_residual else None
        out, pre = room_for(M, N, ld, dtype), room_for(M, N, ld + 8 * (i % 2), dtype)
        zr.mx4_matmul(a, b, out[:, :N], bias=bias, activation=act, residual=residual, pre=pre[:, :N] if has_pre else None)
        (y, e_y), (h, e_h) = expect(av, bv, bias, act, residual, dtype)
        near(out[:, :N], y, e_y, (act, "out"))
        assert bool((out[:, N:] == 7.0).all())
        if has_pre:
            near(pre[:, :N], h, e_h, (act, "pre"))
            assert bool((pre[:, N:] == 7.0).all())
        else:
            assert bool((pre == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(1, 300, 600), (3, 129, 2048), (16, 1000, 513), (17, 40, 100), (2, 20000, 64), (200, 515, 300)])
def test_linear(M, N, K):
    """Few tokens by clusters of every size, and more of them."""
    dtype = (F32, F16, BF16)[M % 3]
    x = matrix(M, K, dtype, seed=M, wide=False)
    xv = ref.values(*ref.quantise(on_host(x)), K)
    _, w, wv = operand(N, K, 2, 1.5 / math.sqrt(K))
    g = torch.Generator().manual_seed(M)
    for i, (act, has_bias, has_residual, has_pre) in enumerate(KINDS):
        out_dtype = (BF16, F32)[i % 2]
        bias = torch.randn(N, generator=g).to((F32, BF16, F16)[i % 3]).cuda() if has_bias else None
        residual = torch.randn(M, N, generator=g).to(out_dtype).cuda() if has_residual else None
        out, pre = room_for(M, N, N + 3, out_dtype), room_for(M, N, N, out_dtype)
        zr.mx4_linear(x, w, out[:, :N], xq=zr.Mx4(M, K) if M > zr.MX4_FEW or i % 2 else None, bias=bias, activation=act, residual=residual,
                      pre=pre if has_pre else None)
        (y, e_y), (h, e_h) = expect(xv, wv, bias, act, residual, out_dtype)
        near(out[:, :N], y, e_y, (act, "out"))
        assert bool((out[:, N:] == 7.0).all())
        if has_pre:
            near(pre, h, e_h, (act, "pre"))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_gradient(M, N, K, dtype):
    _, a, av = operand(M, K, 1, 1.0)
    _, b, bv = operand(N, K, 2, 1.5 / math.sqrt(K))
    s, e = product(av, bv, F32)
    for i, act in enumerate(("relu", "gelu", "silu")):
        ld = (N, N + 5, (N + 15) // 8 * 8)[i]
        pre = room_for(M, N, ld, dtype)
        pre[:, :N] = matrix(M, N, dtype, seed=i, wide=False) * 2
        pre[0, 0] = 0.0
        out = room_for(M, N, (ld, N)[i % 2], dtype)
        zr.mx4_matmul(a, b, out[:, :N], gradient_of=act, pre=pre[:, :N])
        d, e_d = derivative(on_host(pre[:, :N]), act)
        y = s * d
        near(out[:, :N], y, rounded(y, e * np.abs(d) + np.abs(s) * e_d + EPS * np.abs(y) + e * e_d, dtype), act)
        assert bool((out[:, N:] == 7.0).all()) and bool((pre[:, N:] == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(1024, 4096, 1024), (2304, 2304, 512), (2049, 2100, 600)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_pairs_and_many_tiles(M, N, K, dtype):
    """Pairs of blocks, a last round in halves, tiles past both edges: a band of rows and columns at each end in 64 bits, and
    every value against the product without its epilogue."""
    _, a, av = operand(M, K, 1, 1.0)
    _, b, bv = operand(N, K, 2, 1.5 / math.sqrt(K))
    plain = torch.empty(M, N, device="cuda")
    zr.mx4_matmul(a, b, plain)
    bias = torch.randn(N, device="cuda")
    residual = torch.randn(M, N, device="cuda").to(dtype)
    out, pre = torch.empty(M, N, dtype=dtype, device="cuda"), torch.empty(M, N, dtype=dtype, device="cuda")
    zr.mx4_matmul(a, b, out, bias=bias, activation="gelu", residual=residual, pre=pre)
    rows = np.r_[0:40, M - 40:M]
    (y, e_y), (h, e_h) = expect(av[rows], bv, bias, "gelu", residual[rows], dtype)
    near(out[rows], y, e_y, "out")
    near(pre[rows], h, e_h, "pre")
    # the same sums in the same order where the output's type does not choose another form: within the bound of both
    s = plain.double() + bias.double()
    tol = float(e_h.max()) * 2 + (2.0 ** -8 if dtype == BF16 else 0) * s.abs()
    assert bool(((pre.double() - s).abs() <= tol).all())
    dx = torch.empty(M, N, dtype=dtype, device="cuda")
    zr.mx4_matmul(a, b, dx, gradient_of="silu", pre=pre)
    d, e_d = derivative(on_host(pre[rows]), "silu")
    s, e = product(av[rows], bv, F32)
    near(dx[rows], s * d, rounded(s * d, e * np.abs(d) + np.abs(s) * e_d + EPS * np.abs(s * d) + e * e_d, dtype), "gradient")
    assert bool(torch.isfinite(dx).all()) and bool((dx[40:-40].float().abs().amax(1) > 0).all())


@pytest.mark.parametrize("M,N,K", [(3, 300, 600), (64, 520, 8192), (300, 515, 768), (1024, 4096, 1024)])
def test_in_place(M, N, K):
    """The residual, or a gradient's pre, as the output itself: the bytes of a call with an output of its own."""
    _, a, _ = operand(M, K, 1, 1.0)
    _, b, _ = operand(N, K, 2, 1.5 / math.sqrt(K))
    for dtype, ld in ((BF16, N), (F32, N + 3)):
        start = torch.randn(M, ld, device="cuda").to(dtype)
        want, out = torch.empty_like(start), start.clone()
        zr.mx4_matmul(a, b, want[:, :N], activation="silu", residual=start[:, :N])
        zr.mx4_matmul(a, b, out[:, :N], activation="silu", residual=out[:, :N])
        assert torch.equal(out[:, :N], want[:, :N]) and torch.equal(out[:, N:], start[:, N:])
        out.copy_(start)
        zr.mx4_matmul(a, b, want[:, :N], gradient_of="gelu", pre=start[:, :N])
        zr.mx4_matmul(a, b, out[:, :N], gradient_of="gelu", pre=out[:, :N])
        assert torch.equal(out[:, :N], want[:, :N]) and torch.equal(out[:, N:], start[:, N:])


def test_side_by_side():
    """Out, pre and residual as columns of one matrix: rows between each other's rows."""
    M, N, K = 150, 72, 96
    _, a, av = operand(M, K, 1, 1.0)
    _, b, bv = operand(N, K, 2, 0.2)
    room = torch.randn(M, 3 * N, device="cuda")
    residual = room[:, 2 * N:].clone()
    zr.mx4_matmul(a, b, room[:, :N], activation="relu", pre=room[:, N:2 * N], residual=room[:, 2 * N:])
    (y, e_y), (h, e_h) = expect(av, bv, None, "relu", residual, F32)
    near(room[:, :N], y, e_y, "out")
    near(room[:, N:2 * N], h, e_h, "pre")
    assert torch.equal(room[:, 2 * N:], residual)


def test_a_sum_of_nothing():
    bias, residual = torch.randn(30, device="cuda"), torch.randn(5, 30, device="cuda")
    out = torch.empty(5, 30, device="cuda")
    zr.mx4_matmul(zr.Mx4(5, 0), zr.Mx4(30, 0), out, bias=bias, activation="relu", residual=residual)
    assert torch.equal(out, bias.clamp(min=0) + residual)
    zr.mx4_linear(torch.empty(5, 0, device="cuda"), zr.Mx4(30, 0), out, bias=bias, residual=residual)
    assert torch.equal(out, bias + residual)
    zr.mx4_matmul(zr.Mx4(0, 32), zr.Mx4(6, 32), torch.empty(0, 6, device="cuda"), bias=torch.empty(6, device="cuda"))


def test_far_out_values():
    """Activations and derivatives at the ends of the types: no NaN from what overflows on the way."""
    h = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 90.0, -90.0, 1e4, -1e4, 1e19, -1e19, 1e38, -1e38, 3e38, -3e38], device="cuda")
    n = len(h)
    out = torch.empty(1, n, device="cuda")
    for act in ("relu", "gelu", "silu"):
        zr.mx4_matmul(zr.Mx4(1, 0), zr.Mx4(n, 0), out, bias=h, activation=act)
        want, e = activation(on_host(h)[None], np.zeros((1, n)), act)
        near(out, want, e + EPS * np.abs(want) + 2.0 ** -100, act)
    x = torch.zeros(1, 32, device="cuda")
    x[0, 0] = 1.0
    w = torch.zeros(n, 32, device="cuda")
    w[:, 0] = 2.0
    xq, wq = zr.Mx4(1, 32), zr.Mx4(n, 32)
    zr.mx4_quantize(x, xq)
    zr.mx4_quantize(w, wq)
    for act in ("relu", "gelu", "silu"):
        zr.mx4_matmul(xq, wq, out, gradient_of=act, pre=h[None])
        with np.errstate(all="ignore"):
            clipped = np.clip(on_host(h)[None], -300, 300)  # where every derivative has long been 0 or 1
            d, e = derivative(clipped, act)
        near(out, 2 * d, 2 * e + EPS, act)


def test_what_is_no_number_travels():
    """NaN and infinities of the operands, the bias, the residual and pre reach the outputs that they are part of."""
    M, N, K = 40, 50, 64
    x = matrix(M, K, F32, seed=1, wide=False)
    x[3, 5] = NAN
    a, b = zr.Mx4(M, K), operand(N, K, 2, 1.0)[1]
    zr.mx4_quantize(x, a)
    bias, residual = torch.zeros(N, device="cuda"), torch.zeros(M, N, device="cuda")
    bias[7], residual[10, 11] = NAN, NAN
    out, pre = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    for act in (None, "relu", "gelu", "silu"):
        zr.mx4_matmul(a, b, out, bias=bias, activation=act, residual=residual, pre=pre)
        want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        want[3], want[:, 7] = True, True
        assert torch.equal(torch.isnan(pre), want)
        want[10, 11] = True
        assert torch.equal(torch.isnan(out), want), act
    pre = torch.zeros(M, N, device="cuda")
    pre[20, 21] = NAN
    for act in ("relu", "gelu", "silu"):
        zr.mx4_matmul(a, b, out, gradient_of=act, pre=pre)
        want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        want[3], want[20, 21] = True, True
        assert torch.equal(torch.isnan(out), want), act


def test_captured_and_on_another_stream():
    M, N, K = 300, 515, 768
    x = matrix(M, K, BF16, seed=1, wide=False)
    _, w, _ = operand(N, K, 2, 0.05)
    bias, residual, xq = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").bfloat16(), zr.Mx4(M, K)

    def call(o, stream=None):
        zr.mx4_linear(x, w, o[0], xq=xq, stream=stream, bias=bias, activation="gelu", residual=residual, pre=o[1])
        zr.mx4_linear(x[:4], w, o[2], stream=stream, bias=bias, activation="gelu")
        zr.column_sums(o[0], o[3], stream=stream)

    def outputs():
        return [torch.full((M, N), 7.0, dtype=BF16, device="cuda"), torch.full((M, N), 7.0, dtype=BF16, device="cuda"),
                torch.full((4, N), 7.0, dtype=BF16, device="cuda"), torch.full((N,), 7.0, device="cuda")]

    outs = outputs()
    call(outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    x.copy_(x.flip(0))
    plain, side = outputs(), outputs()
    call(plain)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(side, stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(side, plain))


@pytest.mark.parametrize("M,N,K", [(8, 300, 700), (100, 300, 700), (64, 512, 8192), (1024, 4096, 4096)])
def test_waits_end_and_say_so(M, N, K):
    """Few tokens, blocks alone, clusters and pairs with all that an epilogue takes in: a wait that runs out ends the call."""
    x, a, _ = operand(M, K, 1, 1.0)
    _, b, _ = operand(N, K, 2, 1.5 / math.sqrt(K))
    bias, residual = torch.randn(N, device="cuda"), torch.randn(M, N, device="cuda").bfloat16()
    out, pre, xq = torch.empty_like(residual), torch.empty_like(residual), zr.Mx4(M, K)

    def call():
        zr.mx4_linear(x, b, out, xq=xq, bias=bias, activation="gelu", residual=residual, pre=pre)

    call()
    want = out.clone(), pre.clone()
    zr.mx4_status()
    zr.lib().zr_mx4_stall_waits(1)
    try:
        call()
        zr.mx4_matmul(a, b, out, gradient_of="gelu", pre=residual)
        torch.cuda.synchronize()
    finally:
        zr.lib().zr_mx4_stall_waits(0)
    with pytest.raises(zr.ZrError) as e:
        zr.mx4_status()
    assert e.value.status == 5
    call()
    assert torch.equal(out, want[0]) and torch.equal(pre, want[1])
    zr.mx4_status()


def test_a_layer_and_its_gradients_against_differences():
    """y = residual + gelu(x W^T + b) V^T + c in one pass forward and one back, from the 4-bit values: the gradients of the
    bias, of h and of the weights against differences of the loss in 64 bits."""
    T, D, F = 6, 40, 33
    g = torch.Generator().manual_seed(5)
    xv, wv = operand(T, D, 1, 1.0)[2], operand(F, D, 2, 0.3)[2]
    vv, dyv = operand(D, F, 3, 0.3)[2], operand(T, D, 4, 1.0)[2]
    x, w, v, v_t, dy = zr.Mx4(T, D), zr.Mx4(F, D), zr.Mx4(D, F), zr.Mx4(F, D), zr.Mx4(T, D)
    for q, m in ((x, xv), (w, wv), (dy, dyv)):
        zr.mx4_quantize(torch.from_numpy(m).float().cuda(), q)
    zr.mx4_quantize(torch.from_numpy(vv).float().cuda(), v, v_t)
    b = torch.randn(F, generator=g).cuda()
    h, act, dh, db = torch.empty(T, F, device="cuda"), torch.empty(T, F, device="cuda"), torch.empty(T, F, device="cuda"), torch.empty(F, device="cuda")
    zr.mx4_matmul(x, w, act, bias=b, activation="gelu", pre=h)
    zr.mx4_matmul(dy, v_t, dh, gradient_of="gelu", pre=h)
    zr.column_sums(dh, db)
    v_tv = np.empty((F, D))
    back = torch.empty(F, D, device="cuda")
    zr.mx4_dequantize(v_t, back)
    v_tv = on_host(back)  # V as the backward product takes it

    def loss(bias, shift=None):
        pre = xv @ wv.T + bias + (0 if shift is None else shift)
        u, _ = parts(pre, "gelu")
        return (dyv * ((pre * logistic(u)) @ v_tv)).sum()

    b0, step = on_host(b), 1e-5
    for i in range(F):
        up, down = b0.copy(), b0.copy()
        up[i] += step
        down[i] -= step
        slope = (loss(up) - loss(down)) / (2 * step)
        assert abs(float(db[i]) - slope) <= 1e-4 * (abs(slope) + np.abs(on_host(db)).max())
    for t, i in ((0, 0), (3, 7), (5, 32)):
        d = np.zeros((T, F))
        d[t, i] = step
        slope = (loss(b0, d) - loss(b0, -d)) / (2 * step)
        assert abs(float(dh[t, i]) - slope) <= 1e-4 * (abs(slope) + np.abs(on_host(dh)).max())


# ------------------------------------------------------------------ column sums
@pytest.mark.parametrize("M,N", [(1, 1), (3, 5), (63, 64), (700, 130), (5000, 48), (4097, 2048), (8192, 6), (300, 40001)])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_column_sums(M, N, dtype):
    """Sums of M values in fp32: each thread adds its share of the rows, then halves of them, then a cluster's parts; no
    chain is longer than M / 8 + 30 additions."""
    for ld in (N, N + 3, (N + 15) // 8 * 8):
        x = torch.full((M, ld), NAN, dtype=dtype, device="cuda")
        x[:, :N] = torch.randn(M, N, device="cuda").to(dtype)
        room = torch.full((N + 16,), 7.0, device="cuda")
        zr.column_sums(x[:, :N], room[8:8 + N])
        v = on_host(x[:, :N])
        near(room[8:8 + N], v.sum(0), np.abs(v).sum(0) * EPS * (M / 8 + 30), "sums")
        assert bool((room[:8] == 7).all()) and bool((room[8 + N:] == 7).all())


def test_column_sums_of_nothing_and_of_what_is_no_number():
    out = torch.full((9,), 7.0, device="cuda")
    zr.column_sums(torch.empty(0, 9, device="cuda"), out)
    assert bool((out == 0).all())
    x = torch.zeros(100, 9, device="cuda")
    x[50, 3], x[60, 4] = NAN, INF
    zr.column_sums(x, out)
    assert math.isnan(float(out[3])) and float(out[4]) == INF and bool((out[5:] == 0).all())
    zr.column_sums(torch.empty(5, 0, device="cuda"), torch.empty(0, device="cuda"))


def test_column_sums_past_32_bits():
    x = torch.ones(70_001, 32_000, dtype=BF16, device="cuda")
    out = torch.empty(32_000, device="cuda")
    zr.column_sums(x, out)
    assert bool((out == 70_001).all())
