"""What is measured of the 4-bit and distillation operators, and their plain forms.

Four passes, as a program that trains a model towards 4-bit weights from a teacher makes them:

- quantise: a matrix to microscaled 4-bit floating point (E2M1 values, one power-of-two scale for 32 neighbours), by its
  rows or by rows and columns, to nearest or stochastically, and back to the values that it stands for;
- linear: tokens times a 4-bit weight matrix, the tokens quantised in the pass;
- backward: both products of a linear layer's gradient, the gradient quantised both ways in the pass;
- distill: the loss against a teacher's top logits, and its gradient times the loss scale.

A 4-bit matrix lies in memory as tiles of 128 rows and 256 columns of 17,408 bytes: 128 rows of 128 bytes of codes, the
16-byte chunk j of row r at chunk j ^ (r % 8), the lower code of a byte first; then for each half of 128 columns
512 bytes of scales, [row % 32][row // 32][scale]. `pack` and `unpack` state that layout in torch.
"""
import math

import torch

own = False  # False: the plain forms; True: the framework's operators

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK, TILE_R, TILE_C, TILE_BYTES = 32, 128, 256, 17408


def listed():
    return [
        # one attention projection of the 124M shapes, from the fp32 masters, after a step
        {"name": "quantise_projection", "op": "quantise", "rows": 768, "cols": 768, "dtype": "f32", "both": False, "stochastic": False},
        # the 1.3B shapes' embedding, both ways: its rows for the logits, its columns for the gradient behind them
        {"name": "quantise_embedding", "op": "quantise", "rows": 50304, "cols": 2048, "dtype": "f32", "both": True, "stochastic": False},
        # a gradient of a ragged batch, both ways, stochastically, as the two products of a backward pass take it
        {"name": "quantise_gradient", "op": "quantise", "rows": 4099, "cols": 2049, "dtype": "bf16", "both": True, "stochastic": True},
        # serving one token: the first product of the 1.3B shapes' feed-forward
        {"name": "linear_one_token", "op": "linear", "tokens": 1, "k": 2048, "n": 8192, "dtype": "bf16", "out": "bf16"},
        # serving eight requests: the logits in fp32
        {"name": "linear_head_8", "op": "linear", "tokens": 8, "k": 2048, "n": 50304, "dtype": "f16", "out": "f32"},
        # a ragged prompt through a layer whose sizes fit no tile
        {"name": "linear_ragged", "op": "linear", "tokens": 333, "k": 1000, "n": 2309, "dtype": "f32", "out": "f32"},
        # a prompt through the 1.3B shapes' qkv product
        {"name": "linear_prompt", "op": "linear", "tokens": 2048, "k": 2048, "n": 6144, "dtype": "f16", "out": "f16"},
        # a training batch's logits, the largest product there is
        {"name": "linear_head_train", "op": "linear", "tokens": 8192, "k": 2048, "n": 50304, "dtype": "bf16", "out": "bf16"},
        # a training batch through the backward of the 1.3B shapes' second feed-forward product
        {"name": "backward_feed_forward", "op": "backward", "tokens": 8192, "k": 8192, "n": 2048, "dtype": "bf16"},
        # a short ragged batch through the backward of the 124M shapes' qkv product
        {"name": "backward_ragged", "op": "backward", "tokens": 777, "k": 768, "n": 2304, "dtype": "f16"},
        # a training batch's loss over the padded vocabulary
        {"name": "distill_train", "op": "distill", "tokens": 8192, "vocab": 50304, "top": 64, "dtype": "bf16", "temperature": 2.0},
        # a few generated tokens scored against a teacher, fp32 logits, an odd vocabulary
        {"name": "distill_few", "op": "distill", "tokens": 13, "vocab": 50257, "top": 100, "dtype": "f32", "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "linear", "linear", "backward", "distill"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "quantise":
        rows, cols = _log(rng, 1, 50304), _log(rng, 33, 8192)
        rows = max(1, min(rows, 40000 * 2048 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "both": rng.random() < 0.5, "stochastic": rng.random() < 0.5}
    if op == "linear":
        tokens, k, n = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 50304)
        n = max(64, min(n, 8192 * 2048 * 50304 // (tokens * k)))
        return {"op": op, "tokens": tokens, "k": k, "n": n, "dtype": dtype, "out": rng.choice(["f32", "f16", "bf16"])}
    if op == "backward":
        return {"op": op, "tokens": _log(rng, 16, 8192), "k": _log(rng, 256, 8192), "n": _log(rng, 256, 2048), "dtype": rng.choice(["f16", "bf16"])}
    tokens, vocab = _log(rng, 1, 8192), _log(rng, 1000, 150000)
    tokens = max(1, min(tokens, 8192 * 50304 * 2 // (vocab * BYTES[dtype])))
    return {"op": op, "tokens": tokens, "vocab": vocab, "top": _log(rng, 1, 256), "dtype": dtype, "temperature": rng.choice([1.0, 2.0, 4.0])}


# ---------------------------------------------------------------- the 4-bit format, plain, in 32 bits
def _scales(blocks, stochastic):
    """The scale bytes of [..., 32] fp32 values: the power of two under the largest magnitude over 4, 2^(byte - 127)."""
    top = blocks.abs().amax(-1)
    bits = (top.view(torch.int32) >> 23) & 255
    byte = (bits - 2).clamp(min=0)
    if stochastic:  # one power higher where the largest would lie over 6, so that nothing is clipped
        byte = byte + ((top * _power(127 - byte)) > 6)
    return torch.where(bits == 255, 255, byte)


def _power(e):
    """2.0^e for whole e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x):
    """[rows, cols] as fp32 [rows, blocks, 32], zeros behind the last column."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)


def _rounded(x, rand=None):
    """What the rows of x stand for after rounding: (signed values before their scale, scale bytes)."""
    b = _blocks(x)
    byte = _scales(b, rand is not None)
    t = b.abs() * _power(127 - byte.clamp(max=253))[..., None]
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    u = t / step
    if rand is None:
        v = torch.round(u) * step
    else:
        low = torch.floor(u)
        v = (low + ((u - low) > (255.5 - _blocks(rand)) / 256)) * step
    v = torch.copysign(v.clamp(max=6), b)
    return torch.where(byte[..., None] == 255, 0.0, v), byte


def _values(v, byte, cols):
    """Values and scale bytes as the fp32 matrix that they stand for (2^-127, which fp32 holds as a subnormal, in two factors)."""
    out = v * _power(byte.clamp(max=253) - 126)[..., None] * 0.5
    return torch.where(byte[..., None] == 255, math.nan, out).reshape(v.shape[0], -1)[:, :cols]


def _fake(x, rand=None):
    return _values(*_rounded(x, rand), x.shape[1])


def mx4_bytes(rows, cols):
    return -(-rows // TILE_R) * -(-cols // TILE_C) * TILE_BYTES


def pack(v, byte):
    """Signed values [rows, blocks, 32] and scale bytes [rows, blocks] as the bytes of a 4-bit matrix."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    code = torch.bucketize(v.abs(), mag).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    r, nb = byte.shape
    nr, nc = -(-r // TILE_R), -(-nb * BLOCK // TILE_C)
    code = torch.nn.functional.pad(code.view(r, nb * BLOCK), (0, nc * TILE_C - nb * BLOCK, 0, nr * TILE_R - r))
    two = code[:, 0::2] | (code[:, 1::2] << 4)
    two = two.view(nr, TILE_R, nc, 8, 16).permute(0, 2, 1, 3, 4)  # tiles of [row, chunk, byte]
    at = torch.arange(8, device=v.device)[None, :] ^ (torch.arange(TILE_R, device=v.device)[:, None] % 8)
    two = torch.gather(two, 3, at[None, None, :, :, None].expand(nr, nc, TILE_R, 8, 16))  # its own inverse
    sc = torch.nn.functional.pad(byte.to(torch.uint8), (0, nc * 8 - nb, 0, nr * TILE_R - r))
    sc = sc.view(nr, 4, 32, nc, 2, 4).permute(0, 3, 4, 2, 1, 5)  # tiles of [half][row % 32][row // 32][scale]
    return torch.cat([two.reshape(nr, nc, -1), sc.reshape(nr, nc, -1)], 2).reshape(-1).contiguous()


def unpack(data, rows, cols):
    """The fp32 matrix that the bytes of a 4-bit matrix stand for."""
    nr, nc = -(-rows // TILE_R), -(-cols // TILE_C)
    tiles = data.view(nr, nc, TILE_BYTES)
    two = tiles[:, :, :16384].reshape(nr, nc, TILE_R, 8, 16)
    at = torch.arange(8, device=data.device)[None, :] ^ (torch.arange(TILE_R, device=data.device)[:, None] % 8)
    two = torch.gather(two, 3, at[None, None, :, :, None].expand(nr, nc, TILE_R, 8, 16))
    two = two.permute(0, 2, 1, 3, 4).reshape(nr * TILE_R, nc * TILE_C // 2)
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=data.device)
    v = torch.stack([value[(two & 15).int()], value[(two >> 4).int()]], 2).view(nr * TILE_R, -1, BLOCK)
    sc = tiles[:, :, 16384:].reshape(nr, nc, 2, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(nr * TILE_R, -1)
    return _values(v, sc.int(), cols)[:rows]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _tokens(g, rows, cols, dtype):
    """Hidden states: normal, a size for each row, a few channels much larger than the others."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g, device="cuda")] *= 12
    return x.to(DTYPES[dtype])


def _gradient(g, rows, cols, dtype):
    """Gradients under a loss scale: sizes over many powers of two between rows, some rows without any."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    x[torch.rand(rows, generator=g, device="cuda") < 0.05] = 0
    return x.to(DTYPES[dtype])


def _weight(g, rows, cols):
    return 0.02 * torch.randn(rows, cols, generator=g, device="cuda")


def _rand(g, rows, cols):
    return torch.randint(0, 256, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)


def _raw(case, seed):
    """The inputs of a case, in no layout of their own."""
    g, op = _gen(seed), case["op"]
    if op == "quantise":
        r, c = case["rows"], case["cols"]
        x = _weight(g, r, c).to(DTYPES[case["dtype"]]) if not case["stochastic"] else _gradient(g, r, c, case["dtype"])
        return {"x": x, "rand": _rand(g, r, c) if case["stochastic"] else None}
    if op == "linear":
        return {"x": _tokens(g, case["tokens"], case["k"], case["dtype"]), "w": _weight(g, case["n"], case["k"])}
    if op == "backward":
        t, k, n = case["tokens"], case["k"], case["n"]
        return {"x": _tokens(g, t, k, case["dtype"]), "w": _weight(g, n, k), "dy": _gradient(g, t, n, case["dtype"]), "rand": _rand(g, t, n)}
    t, v, top = case["tokens"], case["vocab"], case["top"]
    z = torch.randn(t, v, generator=g, device="cuda")
    z *= 1.5
    first = torch.randint(0, v, (t, 1), generator=g, device="cuda")
    ids = (first + torch.arange(top, device="cuda") * (v // top)) % v  # distinct in a row
    rank = torch.arange(top, device="cuda", dtype=torch.float32)
    teacher = 9 - 1.5 * torch.log1p(rank) + 0.3 * torch.randn(t, top, generator=g, device="cuda")
    z.scatter_(1, ids, 6 - torch.log1p(rank) + torch.randn(t, top, generator=g, device="cuda"))
    kept = torch.randint(0, 2 * top, (t, 1), generator=g, device="cuda")  # half of the rows hold fewer, a few hold none
    ids = torch.where(torch.arange(top, device="cuda") < kept, ids, -1).to(torch.int32)
    weight = (torch.rand(t, generator=g, device="cuda") > 0.1).float() / t  # prompt tokens carry no loss
    return {"z": z.to(DTYPES[case["dtype"]]), "ids": ids, "teacher": teacher, "weight": weight}


LOSS_SCALE = 1024.0


def prepare(case, seed):
    """The inputs on the GPU, the weights in their 4-bit layout, the output buffers that such a program keeps."""
    s = _raw(case, seed)
    s["case"], op = dict(case), case["op"]

    def empty(rows, cols, dtype):
        return torch.empty(rows, cols, dtype=DTYPES[dtype], device="cuda")

    def room(rows, cols):
        return torch.empty(mx4_bytes(rows, cols), dtype=torch.uint8, device="cuda")

    if op == "quantise":
        r, c = case["rows"], case["cols"]
        s["q"], s["out"] = room(r, c), empty(r, c, "bf16")
        if case["both"]:
            s["q_t"], s["out_t"] = room(c, r), empty(c, r, "bf16")
    elif op == "linear":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["w"] = pack(*_rounded(s["w"]))
        s["xq"], s["out"] = room(t, k), empty(t, n, case["out"])
    elif op == "backward":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["w_t"] = pack(*_rounded(s.pop("w").t().contiguous()))  # [k, n], kept from the forward pass
        s["x_t"] = pack(*_rounded(s.pop("x").t().contiguous()))  # [k, tokens], kept from the forward pass
        s["q"], s["q_t"] = room(t, n), room(n, t)
        s["dx"], s["dw"] = empty(t, k, case["dtype"]), empty(n, k, "f32")
    else:
        s["loss"] = torch.empty(case["tokens"], device="cuda")
        s["grad"] = torch.empty_like(s["z"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return (_own if own else _plain)[case["op"]](s, case)


def _plain_quantise(s, case):
    x, rand = s["x"], s["rand"]
    out = [_fake(x, rand).to(torch.bfloat16)]
    if case["both"]:
        out.append(_fake(x.t(), None if rand is None else rand.t()).to(torch.bfloat16))
    return out


def _plain_linear(s, case):
    return (_fake(s["x"]) @ unpack(s["w"], case["n"], case["k"]).t()).to(DTYPES[case["out"]])


def _plain_backward(s, case):
    t, k, n = case["tokens"], case["k"], case["n"]
    dx = _fake(s["dy"], s["rand"]) @ unpack(s["w_t"], k, n).t()
    dw = _fake(s["dy"].t(), s["rand"].t()) @ unpack(s["x_t"], k, t).t()
    return [dx.to(DTYPES[case["dtype"]]), dw]


def _plain_distill(s, case):
    tau, ids, w = case["temperature"], s["ids"].long(), s["weight"]
    z = s["z"].float() / tau
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    kept = ids >= 0
    some = kept.any(1)
    live = (some & (w != 0))[:, None]
    t = torch.where(kept, s["teacher"].float() / tau, -math.inf)
    t = t - torch.where(some[:, None], t.amax(1, keepdim=True), 0.0)
    pe = torch.exp(t)
    p_total = pe.sum(1, keepdim=True)
    p = torch.where(live, pe / p_total, 0.0)
    at = ids.clamp(min=0)
    logs = (t - torch.log(p_total)) - (z.gather(1, at) - torch.log(total))
    loss = w * tau * tau * torch.where(p > 0, p * logs, 0.0).sum(1)
    e /= total
    e.scatter_add_(1, at, -p)
    grad = torch.where(live, e * (w * (tau * LOSS_SCALE))[:, None], 0.0)
    return [loss, grad.to(s["z"].dtype)]


def _own_quantise(s, case):
    import zero_gradient_reduction_gb300 as zr
    r, c = case["rows"], case["cols"]
    q = zr.Mx4(r, c, data=s["q"])
    q_t = zr.Mx4(c, r, data=s["q_t"]) if case["both"] else None
    zr.mx4_quantize(s["x"], q, q_t, rand=s["rand"])
    zr.mx4_dequantize(q, s["out"])
    if q_t is None:
        return [s["out"]]
    zr.mx4_dequantize(q_t, s["out_t"])
    return [s["out"], s["out_t"]]


def _own_linear(s, case):
    import zero_gradient_reduction_gb300 as zr
    w = zr.Mx4(case["n"], case["k"], data=s["w"])
    zr.mx4_linear(s["x"], w, s["out"], xq=zr.Mx4(case["tokens"], case["k"], data=s["xq"]))
    return s["out"]


def _own_backward(s, case):
    import zero_gradient_reduction_gb300 as zr
    t, k, n = case["tokens"], case["k"], case["n"]
    dy, dy_t = zr.Mx4(t, n, data=s["q"]), zr.Mx4(n, t, data=s["q_t"])
    zr.mx4_quantize(s["dy"], dy, dy_t, rand=s["rand"])
    zr.mx4_matmul(dy, zr.Mx4(k, n, data=s["w_t"]), s["dx"])
    zr.mx4_matmul(dy_t, zr.Mx4(k, t, data=s["x_t"]), s["dw"])
    return [s["dx"], s["dw"]]


def _own_distill(s, case):
    import zero_gradient_reduction_gb300 as zr
    zr.distill_topk(s["z"], s["ids"], s["teacher"], s["loss"], s["grad"], weight=s["weight"], temperature=case["temperature"], grad_scale=LOSS_SCALE)
    return [s["loss"], s["grad"]]


_plain = {"quantise": _plain_quantise, "linear": _plain_linear, "backward": _plain_backward, "distill": _plain_distill}
_own = {"quantise": _own_quantise, "linear": _own_linear, "backward": _own_backward, "distill": _own_distill}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    four = 0.5 + 1 / 32  # bytes of a 4-bit value and its share of a scale
    if op == "quantise":
        n, ways = case["rows"] * case["cols"], 2 if case["both"] else 1
        return {"bytes": n * (BYTES[case["dtype"]] + (1 if case["stochastic"] else 0) + ways * (four + 2)), "flops": 2 * n * ways}
    if op == "linear":
        t, k, n = case["tokens"], case["k"], case["n"]
        return {"bytes": t * k * BYTES[case["dtype"]] + n * k * four + t * n * BYTES[case["out"]], "flops": 2 * t * k * n}
    if op == "backward":
        t, k, n = case["tokens"], case["k"], case["n"]
        b = BYTES[case["dtype"]]
        return {"bytes": t * n * (b + 1) + (k * n + k * t) * four + t * k * b + n * k * 4, "flops": 4 * t * k * n}
    t, v = case["tokens"], case["vocab"]
    return {"bytes": t * (2 * v * BYTES[case["dtype"]] + case["top"] * 8 + 8), "flops": 8 * t * v}


# ---------------------------------------------------------------- the definitions in 64 bits
def _two_to(e):
    """2.0^e in 64 bits, from its bits: a power function may be off by a rounding, and values of 16 bits often lie right on a threshold."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx4(x, rand=None):
    """The rows of x as what their 4-bit form stands for: by the thresholds between neighbouring values, in 64 bits."""
    x = x.double()
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, -c % 32)).reshape(r, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)  # frexp's exponent is one over floor(log2)
    if rand is not None:
        e = e + (top * _two_to(-e) > 6)
    t = b.abs() * _two_to(-e)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    out = torch.zeros_like(t)
    if rand is not None:
        u = (torch.nn.functional.pad(rand.double(), (0, -c % 32)).reshape(r, -1, 32) + 0.5) / 256
    for i in range(7):
        lo, hi = grid[i], grid[i + 1]
        if rand is None:  # a tie goes to the value of even index
            mid = (lo + hi) / 2
            over = (t > mid) if i % 2 == 0 else (t >= mid)
        else:
            over = (t - lo) / (hi - lo) > 1 - u
        out = torch.where(over, hi, out)
    return (torch.sign(b) * out * _two_to(e)).reshape(r, -1)[:, :c]


def exact(case, seed):
    s, op = _raw(case, seed), case["op"]
    if op == "quantise":
        out = [_exact_mx4(s["x"], s["rand"])]
        if case["both"]:
            out.append(_exact_mx4(s["x"].t(), None if s["rand"] is None else s["rand"].t()))
        return out
    if op == "linear":
        return _exact_mx4(s["x"]) @ _exact_mx4(s["w"]).t()
    if op == "backward":
        dx = _exact_mx4(s["dy"], s["rand"]) @ _exact_mx4(s["w"].t()).t()
        return [dx, _exact_mx4(s["dy"].t(), s["rand"].t()) @ _exact_mx4(s["x"].t()).t()]
    tau, t, v = case["temperature"], case["tokens"], case["vocab"]
    loss = torch.zeros(t, dtype=torch.float64, device="cuda")
    grad = torch.zeros(t, v, dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 26) // v)
    for a in range(0, t, rows):
        z = torch.log_softmax(s["z"][a:a + rows].double() / tau, 1)
        ids, w = s["ids"][a:a + rows].long(), s["weight"][a:a + rows].double()
        kept = (ids >= 0) & (w != 0)[:, None]
        some = kept.any(1, keepdim=True)
        lp = torch.log_softmax(torch.where(kept, s["teacher"][a:a + rows].double() / tau, -1e300), 1)
        p = torch.where(kept, lp.exp(), 0.0)
        at = ids.clamp(min=0)
        loss[a:a + rows] = w * tau ** 2 * torch.where(kept, p * (lp - z.gather(1, at)), 0.0).sum(1)
        q = torch.where(some, z.exp(), 0.0).scatter_add_(1, at, -p)
        grad[a:a + rows] = q * (w * tau * LOSS_SCALE)[:, None]
    return [loss, grad]
