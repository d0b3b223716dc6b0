"""The post-training losses from their definitions, in numpy and 64 bits, and what fp32 may cost them: used by the tests
alone.

What fp32 may cost. An exponent (z - max) log2(e)/tau carries three roundings (of the parts of the constant, and two of the
multiply-adds) of a term up to A = max |z| log2(e)/tau; exp2 2 units; a sum the roundings of under 100 additions (a
thread's terms by words, threads, warps, blocks) and of under ten rescalings. Each term, and so each sum and each q, is
right to the relative error E = 2^-24 (6 A + 150). A log-probability is one exponent less a logarithm (3 A roundings, E, a
unit of the logarithm and two of its products): 2 E + 2^-24 (6 |logp| + 60)."""
import numpy as np
import torch

EPS = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HALF_ULP = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
SMALLEST = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -134}


def softmax(z, tau):
    """(log q, q) of the rows of z."""
    with np.errstate(invalid="ignore"):
        x = z / tau
        x = x - x.max(1, keepdims=True)
        e = np.exp(x)
        total = e.sum(1, keepdims=True)
        return x - np.log(total), e / total


def relative(z, tau):
    """E, with A of the logits that have a term at all: under the row's maximum by 200 tau they have none."""
    finite = np.where(np.isfinite(z), z, -np.inf)
    counts = finite >= finite.max(1, keepdims=True) - 200 * tau
    return EPS * (6 * np.abs(np.where(counts & np.isfinite(z), z, 0.0)).max(initial=0.0) * 1.45 / tau + 150)


def logp_error(z, tau, logp):
    return 2 * relative(z, tau) + EPS * (6 * np.abs(logp) + 60)


def others(z, tau, a):
    """1 - q at the chosen column, from the other columns."""
    x = z / tau
    x = x - x.max(1, keepdims=True)
    e = np.exp(x)
    total = e.sum(1)
    e[np.arange(len(a)), a] = 0
    return e.sum(1) / total


def gradient(z, tau, a, f):
    """f / tau (1 at a - q), row by row; nothing where f is 0."""
    q = softmax(z, tau)[1]
    g = -q * f[:, None] / tau
    g[np.arange(len(a)), a] = others(z, tau, a) * f / tau
    g[f == 0] = 0
    return g


def gradient_error(z, tau, a, f, df, dtype):
    """E of q (1 - q from its own sum, divided by another: 2 E), the factor's own error and four roundings, then the type's
    (and q under 2^-126, which is none)."""
    with np.errstate(invalid="ignore"):
        share = np.abs(gradient(z, tau, a, np.ones(len(a))))
    rel = 2 * relative(z, tau) + 8 * EPS
    g = share * np.abs(f)[:, None]
    err = g * rel + share * df[:, None] * (1 + rel)
    return err + (g + err) * HALF_ULP[dtype] * (1 + 2.0 ** -10) + SMALLEST[dtype] + 2.0 ** -124 * np.abs(f)[:, None]


def policy(z, a, old, adv, w, lo, hi, ref, kl, tau, scale):
    """((loss, logp, f), their errors): f is dloss/dlogp times scale."""
    T = len(a)
    live = (w != 0) & (a >= 0)
    at, z = np.where(live, a, 0), np.where(live[:, None], z, 0.0)
    logp = np.where(live, softmax(z, tau)[0][np.arange(T), at], 0.0)
    e_lp = logp_error(z, tau, logp)
    with np.errstate(all="ignore"):
        up, e_up = logp - old, e_lp + EPS * 2 * np.abs(logp - old)
        r = np.exp(up)
        clipped = r * adv > np.clip(r, 1 - lo, 1 + hi) * adv
        kept = np.where(clipped, np.clip(r, 1 - lo, 1 + hi), r)
        e_r = np.where(clipped, 4 * EPS * kept, r * (np.expm1(e_up) + 8 * EPS))
        value, e_value = -kept * adv, np.abs(adv) * e_r + 4 * EPS * np.abs(kept * adv)
        slope, e_slope = np.where(clipped, 0.0, -r * adv), np.where(clipped, 0.0, e_value)
        if kl:
            d = ref - logp
            e_d = e_lp + 2 * EPS * np.abs(d)
            more = np.expm1(d)
            e_more = np.exp(d) * np.expm1(e_d) + 4 * EPS * np.abs(more)
            value = value + kl * (more - d)
            e_value = e_value + np.abs(kl) * (e_more + e_d + 8 * EPS * (np.abs(more) + np.abs(d))) + 4 * EPS * np.abs(value)
            slope = slope - kl * more
            e_slope = e_slope + np.abs(kl) * (e_more + 4 * EPS * np.abs(more)) + 4 * EPS * np.abs(slope)
        loss, f = np.where(live, w * value, 0.0), np.where(live, w * scale * slope, 0.0)
        e_loss = np.where(live, np.abs(w) * e_value * (1 + 4 * EPS) + 4 * EPS * np.abs(loss), 0.0) + 2.0 ** -149
        e_f = np.where(live, np.abs(w * scale) * e_slope * (1 + 4 * EPS) + 8 * EPS * np.abs(f), 0.0)
    return (loss, logp, f), (e_loss, np.where(live, e_lp, 0.0), e_f)


def preference(z, a, starts, ref, w, beta, smoothing, tau, scale):
    """((loss, rewards, f of each row, whether it is of a sequence), errors of the first three)."""
    T, pairs = len(a), len(w)
    inside = np.zeros(T, bool)
    rewards, e_rewards = np.zeros(2 * pairs), np.zeros(2 * pairs)
    logp = softmax(z, tau)[0][np.arange(T), np.maximum(a, 0)]
    e_lp = logp_error(z, tau, logp)
    for s in range(2 * pairs):
        rows = np.arange(starts[s], starts[s + 1])
        inside[rows] = True
        rows = rows[a[rows] >= 0]
        if w[s // 2] == 0:
            continue
        rewards[s] = beta * (logp[rows] - ref[rows]).sum()
        e_rewards[s] = abs(beta) * (e_lp[rows] + EPS * np.abs(logp[rows] - ref[rows])).sum() + 4 * EPS * abs(rewards[s])
    m = rewards[0::2] - rewards[1::2]
    e_m = e_rewards[0::2] + e_rewards[1::2] + EPS * np.abs(m)
    log_up, log_down = -np.logaddexp(0, -m), -np.logaddexp(0, m)
    loss = np.where(w == 0, 0.0, -w * ((1 - smoothing) * log_up + smoothing * log_down))
    # the loss rises by at most 1 for 1 of m, the logistic by 1/4; an exponential of m, logarithms, sums and products
    e_loss = np.abs(w) * (e_m * (1 + 2 * EPS) + 16 * EPS * (np.abs(log_up) + np.abs(m) * smoothing)) + 2.0 ** -149
    slope = (1 - smoothing) * np.exp(log_down) - smoothing * np.exp(log_up)
    e_slope = np.minimum(e_m / 4, np.exp(-np.abs(m)) * np.expm1(e_m)) + EPS * (8 * (np.exp(log_down) + smoothing * np.exp(log_up)))
    f, e_f = np.zeros(T), np.zeros(T)
    for s in range(2 * pairs):
        rows = slice(starts[s], starts[s + 1])
        sign = -1.0 if s % 2 == 0 else 1.0
        f[rows] = np.where(a[rows] >= 0, sign * w[s // 2] * beta * scale * slope[s // 2], 0.0)
        e_f[rows] = np.where(a[rows] >= 0, abs(w[s // 2] * beta * scale) * e_slope[s // 2] + 8 * EPS * np.abs(f[rows]), 0.0)
    return (loss, rewards, f, inside), (e_loss, e_rewards, e_f)


def logits(T, V, dtype, g, ld=None, spread=2.0, certain=4.0):
    """(logits on the GPU with row stride ld, chosen columns): some hardly likely, some almost certain."""
    z = torch.randn(T, V, generator=g) * spread
    ids = torch.randint(0, V, (T,), generator=g)
    z[torch.arange(T), ids] += certain * torch.randn(T, generator=g) + certain
    room = torch.zeros(T, ld or V, dtype=dtype, device="cuda")
    room[:, :V] = z.to(dtype).cuda()
    return room[:, :V], ids


def near(got, want, bound, what=""):
    d = np.abs(got.double().cpu().numpy() - want)
    assert (d <= bound).all(), (what, float((d - bound).max()), float(d.max()), np.argwhere(~(d <= bound))[:4])
