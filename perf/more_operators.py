"""What is measured of the post-training losses and of the 4-bit layers around them, and their plain forms.

Five passes, as a program that trains a policy with 4-bit layers from rewards or preferences makes them:

- logprobs: the log-probability of each row's chosen token, and the entropy of its distribution, as the behaviour and the
  reference policy are scored;
- policy: the clipped policy loss with a KL term of each token, and its gradient at the logits times the loss scale;
- preference: the loss of pairs of sequences by their log-probability ratios, and its gradient likewise;
- layer: tokens times a 4-bit weight matrix with bias, activation and residual, the tokens quantised in the pass;
- layer_grad: what such a layer's output gradient, in 4 bits, is before the activation below it, and its bias's gradient.

A 4-bit matrix (E2M1 values, one power-of-two scale for 32 neighbours of a row) lies in memory as tiles of 128 rows and
256 columns of 17,408 bytes: 128 rows of 128 bytes of codes, the 16-byte chunk j of row r at chunk j ^ (r % 8), the lower
code of a byte first; then for each half of 128 columns 512 bytes of scales, [row % 32][row // 32][scale].
"""
import math

import torch

own = False  # False: the plain forms; True: the framework's operators

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK, TILE_R, TILE_C, TILE_BYTES = 32, 128, 256, 17408
LOSS_SCALE = 1024.0
CLIP, KL, BETA, SMOOTHING = (0.2, 0.28), 0.05, 0.1, 0.1


def listed():
    return [
        # a few generated tokens scored by the reference policy, fp32 logits, an odd vocabulary
        {"name": "logprobs_few", "op": "logprobs", "tokens": 13, "vocab": 50257, "dtype": "f32", "entropy": False, "temperature": 1.0},
        # a batch of samples scored with its entropy, over the padded vocabulary
        {"name": "logprobs_batch", "op": "logprobs", "tokens": 8192, "vocab": 50304, "dtype": "bf16", "entropy": True, "temperature": 0.7},
        # the last tokens of one sample, an odd vocabulary
        {"name": "policy_few", "op": "policy", "tokens": 11, "vocab": 50257, "dtype": "f32", "temperature": 1.0},
        # a short ragged batch whose rows fit no 16-byte boundary
        {"name": "policy_ragged", "op": "policy", "tokens": 777, "vocab": 50257, "dtype": "f16", "temperature": 1.0},
        # a training batch over the padded vocabulary, sampled at a temperature
        {"name": "policy_train", "op": "policy", "tokens": 8192, "vocab": 50304, "dtype": "bf16", "temperature": 0.8},
        # one pair of short answers, an odd vocabulary
        {"name": "preference_pair", "op": "preference", "pairs": 1, "tokens": 61, "vocab": 50257, "dtype": "bf16"},
        # a training batch of pairs of ragged lengths over the padded vocabulary
        {"name": "preference_train", "op": "preference", "pairs": 16, "tokens": 8192, "vocab": 50304, "dtype": "bf16"},
        # serving one token: the first product of the 1.3B shapes' feed-forward, with its bias and activation
        {"name": "layer_one_token", "op": "layer", "tokens": 1, "k": 2048, "n": 8192, "dtype": "bf16", "activation": "gelu", "residual": False, "keep": False},
        # a ragged prompt through a layer whose sizes fit no tile
        {"name": "layer_ragged", "op": "layer", "tokens": 333, "k": 1000, "n": 2309, "dtype": "f32", "activation": "silu", "residual": True, "keep": False},
        # a training batch through the first product of the 1.3B shapes' feed-forward, what its backward needs kept
        {"name": "layer_train", "op": "layer", "tokens": 8192, "k": 2048, "n": 8192, "dtype": "bf16", "activation": "gelu", "residual": False, "keep": True},
        # the same batch back through the second product of it, to the first's output before the activation
        {"name": "layer_grad_train", "op": "layer_grad", "tokens": 8192, "k": 8192, "n": 2048, "dtype": "bf16", "activation": "gelu"},
        # a short ragged batch back through the 124M shapes' feed-forward at half its width
        {"name": "layer_grad_ragged", "op": "layer_grad", "tokens": 777, "k": 1536, "n": 768, "dtype": "f16", "activation": "relu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "policy", "preference", "preference", "layer", "layer", "layer_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op in ("layer", "layer_grad"):
        tokens, k, n = _log(rng, 1, 8192), _log(rng, 64, 8192), _log(rng, 64, 8192)
        n = max(64, min(n, 8192 * 2048 * 8192 // (tokens * k)))
        case = {"op": op, "tokens": tokens, "k": k, "n": n, "dtype": dtype, "activation": rng.choice(["none", "relu", "gelu", "silu"])}
        if op == "layer":
            case.update(residual=rng.random() < 0.5, keep=rng.random() < 0.3)
        elif case["activation"] == "none":
            case["activation"] = "gelu"
        return case
    tokens, vocab = _log(rng, 1, 8192), _log(rng, 1000, 150000)
    tokens = max(1, min(tokens, 8192 * 50304 * 2 // (vocab * BYTES[dtype])))
    if op == "preference":
        return {"op": op, "pairs": max(1, min(_log(rng, 1, 64), tokens // 2)), "tokens": tokens, "vocab": vocab, "dtype": dtype}
    case = {"op": op, "tokens": tokens, "vocab": vocab, "dtype": dtype, "temperature": rng.choice([0.6, 1.0, 1.5])}
    if op == "logprobs":
        case["entropy"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- the 4-bit format, plain, in 32 bits
def _power(e):
    """2.0^e for whole e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _rounded(x):
    """What the rows of x stand for after rounding to nearest: (signed values before their scale [rows, blocks, 32],
    scale bytes [rows, blocks]), zeros behind the last column. A scale is the power of two under the block's largest
    magnitude over 4, 2^(byte - 127)."""
    x = x.float()
    b = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).view(x.shape[0], -1, BLOCK)
    byte = (((b.abs().amax(-1).view(torch.int32) >> 23) & 255) - 2).clamp(min=0)
    t = b.abs() * _power(127 - byte)[..., None]
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    return torch.copysign((torch.round(t / step) * step).clamp(max=6), b), byte


def _values(v, byte, cols):
    """Values and scale bytes as the fp32 matrix that they stand for."""
    return (v * _power(byte - 126)[..., None] * 0.5).reshape(v.shape[0], -1)[:, :cols]


def mx4_bytes(rows, cols):
    return -(-rows // TILE_R) * -(-cols // TILE_C) * TILE_BYTES


def _chunks(tiles):
    """Chunk j of row r and chunk j ^ (r % 8) of [.., .., 128, 8, 16] exchanged: its own inverse."""
    at = torch.arange(8, device=tiles.device)[None, :] ^ (torch.arange(TILE_R, device=tiles.device)[:, None] % 8)
    return torch.gather(tiles, 3, at[None, None, :, :, None].expand_as(tiles))


def pack(v, byte):
    """Signed values [rows, blocks, 32] and scale bytes [rows, blocks] as the bytes of a 4-bit matrix."""
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=v.device)
    code = torch.bucketize(v.abs(), mag).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    r, nb = byte.shape
    nr, nc = -(-r // TILE_R), -(-nb * BLOCK // TILE_C)
    code = torch.nn.functional.pad(code.view(r, nb * BLOCK), (0, nc * TILE_C - nb * BLOCK, 0, nr * TILE_R - r))
    two = _chunks((code[:, 0::2] | (code[:, 1::2] << 4)).view(nr, TILE_R, nc, 8, 16).permute(0, 2, 1, 3, 4))
    sc = torch.nn.functional.pad(byte.to(torch.uint8), (0, nc * 8 - nb, 0, nr * TILE_R - r))
    sc = sc.view(nr, 4, 32, nc, 2, 4).permute(0, 3, 4, 2, 1, 5)  # tiles of [half][row % 32][row // 32][scale]
    return torch.cat([two.reshape(nr, nc, -1), sc.reshape(nr, nc, -1)], 2).reshape(-1).contiguous()


def unpack(data, rows, cols):
    """The fp32 matrix that the bytes of a 4-bit matrix stand for."""
    nr, nc = -(-rows // TILE_R), -(-cols // TILE_C)
    tiles = data.view(nr, nc, TILE_BYTES)
    two = _chunks(tiles[:, :, :16384].reshape(nr, nc, TILE_R, 8, 16)).permute(0, 2, 1, 3, 4).reshape(nr * TILE_R, nc * TILE_C // 2)
    value = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=data.device)
    v = torch.stack([value[(two & 15).int()], value[(two >> 4).int()]], 2).view(nr * TILE_R, -1, BLOCK)
    sc = tiles[:, :, 16384:].reshape(nr, nc, 2, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(nr * TILE_R, -1)
    return _values(v, sc.int(), cols)[:rows]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, rows, cols, dtype):
    """Hidden states: normal, a size for each row, a few channels much larger than the others."""
    x = _normal(g, rows, cols)
    x *= torch.exp(0.5 * _normal(g, rows, 1))
    x[:, torch.randint(0, cols, (max(1, cols // 200),), generator=g, device="cuda")] *= 12
    return x.to(DTYPES[dtype])


def _logits(g, tokens, vocab, dtype):
    """(logits, sampled tokens): from hardly likely to almost certain ones."""
    z = _normal(g, tokens, vocab)
    z *= 1.5
    ids = torch.randint(0, vocab, (tokens, 1), generator=g, device="cuda")
    z.scatter_(1, ids, 9 + 3 * _normal(g, tokens, 1))
    return z.to(DTYPES[dtype]), ids[:, 0]


def _scored(z, ids, tau):
    """log softmax(z / tau) at ids in 64 bits, a slice of rows at a time; 0 for ids under 0."""
    out = torch.zeros(z.shape[0], dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 26) // z.shape[1])
    for a in range(0, z.shape[0], rows):
        y = z[a:a + rows].double() / tau
        at = ids[a:a + rows].clamp(min=0)
        lp = y.gather(1, at[:, None])[:, 0] - torch.logsumexp(y, 1)
        out[a:a + rows] = torch.where(ids[a:a + rows] < 0, 0.0, lp)
    return out


def _starts(case, seed):
    """Where each sequence begins: ragged lengths that fill the rows."""
    n, t = 2 * case["pairs"], case["tokens"]
    share = torch.rand(n, generator=torch.Generator().manual_seed(int(seed) + 5), dtype=torch.float64) + 0.3
    at = torch.cumsum(share, 0) / share.sum() * t
    return [0] + [int(v) for v in at[:-1]] + [t]


def _raw(case, seed):
    """The inputs of a case, in no layout of their own."""
    g, op = _gen(seed), case["op"]
    if op == "layer":
        t, k, n = case["tokens"], case["k"], case["n"]
        s = {"x": _tokens(g, t, k, case["dtype"]), "w": 0.02 * _normal(g, n, k), "bias": 0.3 * _normal(g, n)}
        s["residual"] = (2 * _normal(g, t, n)).to(DTYPES[case["dtype"]]) if case["residual"] else None
        return s
    if op == "layer_grad":
        t, k, n = case["tokens"], case["k"], case["n"]
        dy = _normal(g, t, n)  # under a loss scale: sizes over many powers of two between rows, some rows without any
        dy *= torch.exp(_normal(g, t, 1))
        dy[torch.rand(t, generator=g, device="cuda") < 0.05] = 0
        return {"dy": dy.to(DTYPES[case["dtype"]]), "w": 0.02 * _normal(g, n, k), "pre": (1.5 * _normal(g, t, k)).to(DTYPES[case["dtype"]])}
    t, v = case["tokens"], case["vocab"]
    z, ids = _logits(g, t, v, case["dtype"])
    s = {"z": z, "ids": ids}
    if op == "logprobs":
        ids[torch.rand(t, generator=g, device="cuda") < 0.1] = -1  # padding
        return s
    if op == "policy":
        lp = _scored(z, ids, case["temperature"])
        step = 0.2 * torch.randn(t, generator=g, device="cuda", dtype=torch.float64)  # the policy's, since the sample
        for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):  # where the gradient jumps, no two roundings agree
            step = torch.where((step - border).abs() < 1e-3, border + 2e-3, step)
        s["old"] = (lp - step).float()
        s["ref"] = (lp - 0.3 * torch.randn(t, generator=g, device="cuda", dtype=torch.float64)).float()
        s["advantage"] = _normal(g, t)
        s["weight"] = (torch.rand(t, generator=g, device="cuda") > 0.1).float() / t  # prompt tokens carry no loss
        return s
    starts = _starts(case, seed)
    for a, b in zip(starts[:-1], starts[1:]):
        ids[a:a + (b - a) // 4] = -1  # the prompt
    s["ref"] = (_scored(z, ids, 1.0) + 0.3 * torch.randn(t, generator=g, device="cuda", dtype=torch.float64)).float()
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["weight"] = torch.full((case["pairs"],), 1.0 / case["pairs"], device="cuda")
    return s


def prepare(case, seed):
    """The inputs on the GPU, the weights in their 4-bit layout, the output buffers that such a program keeps."""
    s = _raw(case, seed)
    s["case"], op = dict(case), case["op"]

    def empty(*shape, dtype="f32"):
        return torch.empty(*shape, dtype=DTYPES[dtype], device="cuda")

    if op == "layer":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["w"] = pack(*_rounded(s["w"]))
        s["xq"] = torch.empty(mx4_bytes(t, k), dtype=torch.uint8, device="cuda")
        s["out"] = empty(t, n, dtype=case["dtype"])
        s["pre"] = empty(t, n, dtype=case["dtype"]) if case["keep"] else None
    elif op == "layer_grad":
        t, k, n = case["tokens"], case["k"], case["n"]
        s["w_t"] = pack(*_rounded(s.pop("w").t().contiguous()))  # [k, n], kept from the forward pass
        s["dyq"] = pack(*_rounded(s["dy"]))  # as the weight's gradient takes it too
        s["out"], s["db"] = empty(t, k, dtype=case["dtype"]), empty(n)
    elif op == "logprobs":
        s["logp"] = empty(case["tokens"])
        s["entropy"] = empty(case["tokens"]) if case["entropy"] else None
    else:
        s["grad"] = torch.empty_like(s["z"])
        if op == "policy":
            s["loss"], s["logp"] = empty(case["tokens"]), empty(case["tokens"])
        else:
            s["loss"], s["rewards"] = empty(case["pairs"]), empty(2 * case["pairs"])
            if own:
                import zero_gradient_reduction_gb300 as zr
                s["work"] = torch.empty(zr.preference_bytes(case["tokens"], case["pairs"]), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    return (_own if own else _plain)[case["op"]](s, case)


def _softmax(z, tau):
    """(z / tau less its maximum, its exponentials, their sum) in 32 bits."""
    z = z.float() / tau
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    return z, e, e.sum(1, keepdim=True)


def _plain_logprobs(s, case):
    z, e, total = _softmax(s["z"], case["temperature"])
    on = s["ids"] >= 0
    logp = z.gather(1, s["ids"].clamp(min=0)[:, None])[:, 0] - torch.log(total[:, 0])
    out = [torch.where(on, logp, 0.0)]
    if case["entropy"]:
        out.append(torch.where(on, torch.log(total[:, 0]) - (e * z).sum(1) / total[:, 0], 0.0))
    return out


def _gradient(z, ids, e, total, f):
    """f (1 at the chosen token - softmax), a row each, in the logits' type."""
    grad = e * (-f[:, None] / total)
    grad.scatter_add_(1, ids[:, None], f[:, None])
    return grad.to(z.dtype)


def _plain_policy(s, case):
    tau, w, adv = case["temperature"], s["weight"], s["advantage"]
    z, e, total = _softmax(s["z"], tau)
    logp = z.gather(1, s["ids"][:, None])[:, 0] - torch.log(total[:, 0])
    ratio = torch.exp(logp - s["old"])
    kept = torch.minimum(torch.maximum(ratio, torch.tensor(1 - CLIP[0], device="cuda")), torch.tensor(1 + CLIP[1], device="cuda"))
    far = s["ref"] - logp
    loss = w * (KL * (torch.exp(far) - far - 1) - torch.minimum(ratio * adv, kept * adv))
    slope = torch.where(ratio * adv <= kept * adv, -ratio * adv, 0.0) + KL * (1 - torch.exp(far))
    live = w != 0
    f = torch.where(live, w * slope * (LOSS_SCALE / tau), 0.0)
    return [torch.where(live, loss, 0.0), torch.where(live, logp, 0.0), _gradient(s["z"], s["ids"], e, total, f)]


def _plain_preference(s, case):
    z, e, total = _softmax(s["z"], 1.0)
    on, at = s["ids"] >= 0, s["ids"].clamp(min=0)
    ratio = torch.where(on, z.gather(1, at[:, None])[:, 0] - torch.log(total[:, 0]) - s["ref"], 0.0)
    sequence = torch.searchsorted(s["starts"].long(), torch.arange(case["tokens"], device="cuda"), right=True) - 1
    rewards = BETA * torch.zeros(2 * case["pairs"], dtype=torch.float64, device="cuda").index_add_(0, sequence, ratio.double())
    rewards = rewards.float()
    margin = rewards[0::2] - rewards[1::2]
    up, down = 1 / (1 + torch.exp(-margin)), 1 / (1 + torch.exp(margin))
    soft = torch.log1p(torch.exp(-margin.abs())) + (-margin).clamp(min=0)  # -log of `up`
    loss = s["weight"] * (soft + SMOOTHING * margin)
    slope = s["weight"] * BETA * LOSS_SCALE * (SMOOTHING * up - (1 - SMOOTHING) * down)
    f = torch.stack([slope, -slope], 1).reshape(-1)[sequence]
    return [loss, rewards, _gradient(s["z"], at, e, total, torch.where(on, f, 0.0))]


def _activated(h, name):
    if name == "relu":
        return h.clamp(min=0)
    if name == "gelu":
        return 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))
    return h / (1 + torch.exp(-h)) if name == "silu" else h


def _plain_layer(s, case):
    x = _values(*_rounded(s["x"]), case["k"])
    h = x @ unpack(s["w"], case["n"], case["k"]).t() + s["bias"]
    y = _activated(h, case["activation"])
    if case["residual"]:
        y = y + s["residual"].float()
    out = [y.to(DTYPES[case["dtype"]])]
    return out + [h.to(DTYPES[case["dtype"]])] if case["keep"] else out


def _slope(h, name):
    """The derivative of the activation."""
    if name == "relu":
        return (h > 0).to(h.dtype)
    if name == "gelu":
        t = torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h))
        return 0.5 * (1 + t) + 0.5 * h * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * h * h)
    up = 1 / (1 + torch.exp(-h))
    return up * (1 + h * (1 - up))


def _plain_layer_grad(s, case):
    t, k, n = case["tokens"], case["k"], case["n"]
    dx = unpack(s["dyq"], t, n) @ unpack(s["w_t"], k, n).t()
    return [(dx * _slope(s["pre"].float(), case["activation"])).to(DTYPES[case["dtype"]]), s["dy"].double().sum(0).float()]


def _own_logprobs(s, case):
    import zero_gradient_reduction_gb300 as zr
    zr.token_logprobs(s["z"], s["ids"], s["logp"], entropy=s["entropy"], temperature=case["temperature"])
    return [s["logp"], s["entropy"]] if case["entropy"] else [s["logp"]]


def _own_policy(s, case):
    import zero_gradient_reduction_gb300 as zr
    zr.policy_loss(s["z"], s["ids"], s["old"], s["advantage"], s["loss"], s["grad"], weight=s["weight"], clip=CLIP, ref_logp=s["ref"], kl=KL,
                   logp=s["logp"], temperature=case["temperature"], grad_scale=LOSS_SCALE)
    return [s["loss"], s["logp"], s["grad"]]


def _own_preference(s, case):
    import zero_gradient_reduction_gb300 as zr
    zr.preference_loss(s["z"], s["ids"], s["starts"], s["ref"], s["loss"], s["work"], s["grad"], weight=s["weight"], beta=BETA,
                       smoothing=SMOOTHING, rewards=s["rewards"], grad_scale=LOSS_SCALE)
    return [s["loss"], s["rewards"], s["grad"]]


def _own_layer(s, case):
    import zero_gradient_reduction_gb300 as zr
    w, xq = zr.Mx4(case["n"], case["k"], data=s["w"]), zr.Mx4(case["tokens"], case["k"], data=s["xq"])
    activation = None if case["activation"] == "none" else case["activation"]
    zr.mx4_linear(s["x"], w, s["out"], xq=xq, bias=s["bias"], activation=activation, residual=s["residual"], pre=s["pre"])
    return [s["out"], s["pre"]] if case["keep"] else [s["out"]]


def _own_layer_grad(s, case):
    import zero_gradient_reduction_gb300 as zr
    t, k, n = case["tokens"], case["k"], case["n"]
    zr.mx4_matmul(zr.Mx4(t, n, data=s["dyq"]), zr.Mx4(k, n, data=s["w_t"]), s["out"], gradient_of=case["activation"], pre=s["pre"])
    zr.column_sums(s["dy"], s["db"])
    return [s["out"], s["db"]]


_plain = {"logprobs": _plain_logprobs, "policy": _plain_policy, "preference": _plain_preference, "layer": _plain_layer, "layer_grad": _plain_layer_grad}
_own = {"logprobs": _own_logprobs, "policy": _own_policy, "preference": _own_preference, "layer": _own_layer, "layer_grad": _own_layer_grad}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    four = 0.5 + 1 / 32  # bytes of a 4-bit value and its share of a scale
    if op in ("layer", "layer_grad"):
        t, k, n = case["tokens"], case["k"], case["n"]
        if op == "layer":
            return {"bytes": t * k * b + n * k * four + t * n * b * (1 + case["residual"] + case["keep"]) + 4 * n, "flops": 2 * t * k * n}
        return {"bytes": t * n * (four + b) + k * n * four + 2 * t * k * b + 4 * n, "flops": 2 * t * k * n}
    t, v = case["tokens"], case["vocab"]
    if op == "logprobs":  # a tenth of the rows is padding
        return {"bytes": t * (0.9 * v * b + 12 + 4 * case["entropy"]), "flops": (4 + 2 * case["entropy"]) * t * v}
    if op == "policy":  # a tenth carries no weight
        return {"bytes": t * (1.9 * v * b + 32), "flops": 8 * t * v}
    return {"bytes": t * (1.75 * v * b + 12), "flops": 8 * t * v}  # a quarter is prompt


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_mx4(x):
    """The rows of x as what their 4-bit form stands for: by the thresholds between neighbouring values, in 64 bits."""
    x = x.double()
    r, c = x.shape
    b = torch.nn.functional.pad(x, (0, -c % 32)).reshape(r, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)  # frexp's exponent is one over floor(log2)
    scale = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e from its bits, exactly
    t = b.abs() / scale
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    out = torch.zeros_like(t)
    for i in range(7):
        mid = (grid[i] + grid[i + 1]) / 2  # a tie goes to the value of even index
        out = torch.where((t > mid) if i % 2 == 0 else (t >= mid), grid[i + 1], out)
    return (torch.sign(b) * out * scale).reshape(r, -1)[:, :c]


def _sigmoid(u):
    return torch.where(u >= 0, 1 / (1 + torch.exp(-u.abs())), torch.exp(-u.abs()) / (1 + torch.exp(-u.abs())))


def _exact_activation(h, name):
    """(value, derivative)"""
    if name == "none":
        return h, torch.ones_like(h)
    if name == "relu":
        return torch.where(h > 0, h, 0.0), torch.where(h > 0, 1.0, 0.0).double()
    c = math.sqrt(8 / math.pi) if name == "gelu" else 1.0  # gelu: h sigmoid(2 u) with its tanh's argument u
    cubic = 0.044715 if name == "gelu" else 0.0
    up = _sigmoid(c * (h + cubic * h ** 3))
    return h * up, up + h * up * (1 - up) * c * (1 + 3 * cubic * h ** 2)


def _exact_gradient(s, f, tau):
    """f / tau (1 at the chosen token - softmax(z / tau)) in 64 bits, in slices of rows."""
    z, at = s["z"], s["ids"].clamp(min=0)
    out = torch.empty(z.shape, dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 26) // z.shape[1])
    for a in range(0, z.shape[0], rows):
        q = torch.softmax(z[a:a + rows].double() / tau, 1)
        q.scatter_add_(1, at[a:a + rows, None], -torch.ones_like(q[:, :1]))
        out[a:a + rows] = q * (-f[a:a + rows, None] / tau)
    return out


def exact(case, seed):
    s, op = _raw(case, seed), case["op"]
    if op == "layer":
        h = _exact_mx4(s["x"]) @ _exact_mx4(s["w"]).t() + s["bias"].double()
        y = _exact_activation(h, case["activation"])[0]
        if case["residual"]:
            y = y + s["residual"].double()
        return [y, h] if case["keep"] else [y]
    if op == "layer_grad":
        dx = _exact_mx4(s["dy"]) @ _exact_mx4(s["w"].t()).t()
        return [dx * _exact_activation(s["pre"].double(), case["activation"])[1], s["dy"].double().sum(0)]
    if op == "logprobs":
        tau, out = case["temperature"], [_scored(s["z"], s["ids"], case["temperature"])]
        if case["entropy"]:
            h, rows = torch.zeros(case["tokens"], dtype=torch.float64, device="cuda"), max(1, (1 << 26) // case["vocab"])
            for a in range(0, case["tokens"], rows):
                lq = torch.log_softmax(s["z"][a:a + rows].double() / tau, 1)
                h[a:a + rows] = torch.where(s["ids"][a:a + rows] < 0, 0.0, -(lq.exp() * lq).sum(1))
            out.append(h)
        return out
    if op == "policy":
        tau, w, adv = case["temperature"], s["weight"].double(), s["advantage"].double()
        logp = _scored(s["z"], torch.where(w == 0, -1, s["ids"]), tau)
        up, far = logp - s["old"].double(), s["ref"].double() - logp
        lo, hi = math.log1p(-CLIP[0]), math.log1p(CLIP[1])
        free = torch.where(adv >= 0, up <= hi, up >= lo)  # where the ratio itself is the smaller product
        value = torch.exp(torch.where(free, up, torch.where(adv >= 0, hi, lo)))
        loss = w * (KL * (torch.expm1(far) - far) - value * adv)
        f = w * (torch.where(free, -value * adv, 0.0) - KL * torch.expm1(far)) * LOSS_SCALE
        return [loss, logp, _exact_gradient(s, f, tau)]
    ratio = torch.where(s["ids"] < 0, 0.0, _scored(s["z"], s["ids"], 1.0) - s["ref"].double())
    starts = s["starts"].tolist()
    rewards = torch.stack([BETA * ratio[a:b].sum() for a, b in zip(starts[:-1], starts[1:])])
    margin = rewards[0::2] - rewards[1::2]
    w, up = s["weight"].double(), _sigmoid(margin)
    loss = -w * ((1 - SMOOTHING) * torch.nn.functional.logsigmoid(margin) + SMOOTHING * torch.nn.functional.logsigmoid(-margin))
    slope = w * BETA * LOSS_SCALE * (up - (1 - SMOOTHING))
    f = torch.zeros(case["tokens"], dtype=torch.float64, device="cuda")
    for i, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        f[a:b] = slope[i // 2] if i % 2 == 0 else -slope[i // 2]
    return [loss, rewards, _exact_gradient(s, torch.where(s["ids"] < 0, 0.0, f), 1.0)]
