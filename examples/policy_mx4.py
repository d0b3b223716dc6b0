"""Post-training a small 4-bit network from rewards or from preferences, with the layers, the losses and the ZeRO step together.

The network is a residual block and an output layer on fixed hidden states X: H = gelu(X W1^T + b1), Y = X + H W2^T + b2,
logits = Y E^T, with the fp32 masters in a plan's state. Each step quantises them, runs the block with bias, activation and
residual in the products' epilogues, takes the loss with its gradient times the plan's loss scale in place of the logits,
and goes back: the gradient quantised by chance, dY and dE; the bias's sums; the product behind the activation; dW2, dW1.
The gradients go straight into the replica that the step reduces; one that overflows makes it skip and halve the scale.

With --loss policy tokens are sampled, scored by the policy as it is and by the reference it began as, and trained on twice
with the clipped loss; with --loss preference pairs of sequences are trained on against the reference.

    python examples/policy_mx4.py [--loss policy --tokens 1024 --dim 256 --hidden 512 --vocab 2000 --steps 30]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_gradient_reduction_gb300 as zr  # noqa: E402

BF16 = torch.bfloat16


class Network:
    """The masters, their 4-bit forms both ways, and what a pass keeps for its backward."""

    def __init__(self, tokens, dim, hidden, vocab, generator):
        self.g, self.T = generator, tokens
        self.shapes = {"w1": (hidden, dim), "b1": (hidden,), "w2": (dim, hidden), "b2": (dim,), "e": (vocab, dim)}
        numels = [torch.Size(s).numel() for s in self.shapes.values()]
        self.plan = zr.Plan(numels, W=1, dtype=zr.BF16, stage=1, cap=sum(numels) + 64, fp32_grads=True,
                            scaler=zr.Scaler(init_scale=1024.0, dynamic=True))
        self.state, self.live = self.plan.new_state(), 0
        self.grads = [torch.zeros(self.plan.numel, device="cuda")]
        self.state.master[0].zero_()
        for name, scale in (("w1", dim ** -0.5), ("w2", hidden ** -0.5), ("e", 2 * dim ** -0.5)):
            self.of(self.state.master[0], name).normal_(0, scale, generator=generator)
        zr.all_gather(self.state.master[0], [self.state.param[0]])

        def both(rows, cols):
            return zr.Mx4(rows, cols), zr.Mx4(cols, rows)

        self.w1, self.w2, self.e = both(hidden, dim), both(dim, hidden), both(vocab, dim)
        self.x4, self.h4, self.y4 = both(tokens, dim), both(tokens, hidden), both(tokens, dim)
        self.dz4, self.dy4, self.dh4 = both(tokens, vocab), both(tokens, dim), both(tokens, hidden)

        def empty(cols):
            return torch.empty(tokens, cols, dtype=BF16, device="cuda")

        self.pre, self.h, self.y, self.z = empty(hidden), empty(hidden), empty(dim), empty(vocab)
        self.dy, self.dh = empty(dim), empty(hidden)
        self.rand = {c: torch.empty(tokens, c, dtype=torch.uint8, device="cuda") for c in (vocab, dim, hidden)}

    def of(self, flat, name):
        i = list(self.shapes).index(name)
        at, shape = int(self.plan.tensor_offsets[i]), self.shapes[name]
        return flat[at:at + torch.Size(shape).numel()].view(shape)

    def master(self, name):
        return self.of(self.state.live(self.live)["master"], name)

    def grad(self, name):
        return self.of(self.grads[0], name)

    def forward(self, x):
        """The logits of hidden states x."""
        for name, q in (("w1", self.w1), ("w2", self.w2), ("e", self.e)):
            zr.mx4_quantize(self.master(name), *q)
        zr.mx4_quantize(x, *self.x4)
        zr.mx4_matmul(self.x4[0], self.w1[0], self.h, bias=self.master("b1"), activation="gelu", pre=self.pre)
        zr.mx4_quantize(self.h, *self.h4)
        zr.mx4_matmul(self.h4[0], self.w2[0], self.y, bias=self.master("b2"), residual=x)
        zr.mx4_quantize(self.y, *self.y4)
        zr.mx4_matmul(self.y4[0], self.e[0], self.z)
        return self.z

    def backward(self, dz):
        """The gradients of all masters from the logits' gradient."""
        def quantised(d, q):
            r = self.rand[d.shape[1]]
            r.random_(0, 256, generator=self.g)
            zr.mx4_quantize(d, *q, rand=r)

        quantised(dz, self.dz4)
        zr.mx4_matmul(self.dz4[0], self.e[1], self.dy)
        zr.mx4_matmul(self.dz4[1], self.y4[1], self.grad("e"))
        quantised(self.dy, self.dy4)
        zr.column_sums(self.dy, self.grad("b2"))
        zr.mx4_matmul(self.dy4[1], self.h4[1], self.grad("w2"))
        zr.mx4_matmul(self.dy4[0], self.w2[1], self.dh, gradient_of="gelu", pre=self.pre)
        quantised(self.dh, self.dh4)
        zr.column_sums(self.dh, self.grad("b1"))
        zr.mx4_matmul(self.dh4[1], self.x4[1], self.grad("w1"))

    def step(self, hyper):
        rep = self.plan.step(self.grads, self.state, hyper, report=True)
        self.live = rep.current
        return rep


def train(loss="policy", tokens=1024, dim=256, hidden=512, vocab=2000, steps=30, seed=0, report=print):
    """Mean reward, or mean loss, of each step."""
    length = 16  # of a sequence of a pair
    if loss == "preference" and tokens < 2 * length:
        raise ValueError(f"a pair of sequences has {2 * length} tokens, not {tokens}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    net, hyper = Network(tokens, dim, hidden, vocab, g), zr.AdamW(lr=1e-3, weight_decay=0.0)
    x = torch.randn(tokens, dim, generator=g, device="cuda").to(BF16)
    weight = torch.full((tokens,), 1.0 / tokens, device="cuda")
    out, logp, old, ref = (torch.empty(tokens, device="cuda") for _ in range(4))
    first = net.forward(x).clone()  # the reference's logits
    history = []
    if loss == "preference":
        pairs = tokens // (2 * length)
        starts = torch.arange(0, 2 * pairs + 1, dtype=torch.int32, device="cuda") * length
        ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        ids[::length] = -1  # a prompt token each
        zr.token_logprobs(first, ids, ref)
        work = torch.empty(zr.preference_bytes(tokens, pairs), dtype=torch.uint8, device="cuda")
        each, of_pair = torch.empty(pairs, device="cuda"), torch.full((pairs,), 1.0 / pairs, device="cuda")
    for step in range(steps):
        if loss == "preference":
            z = net.forward(x)
            z[2 * length * pairs:] = 0  # rows of no pair have no gradient
            zr.preference_loss(z, ids, starts, ref, each, work, grad=z, weight=of_pair, beta=0.1, plan=net.plan)
            net.backward(z)
            rep = net.step(hyper)
            history.append(float(each.sum()))
        else:
            z = net.forward(x)
            ids = torch.multinomial(torch.softmax(z.float(), 1), 1, generator=g)[:, 0]
            reward = (ids % 7 == 0).float()
            advantage = (reward - reward.mean()) / (reward.std() + 1e-6)
            zr.token_logprobs(z, ids, old)
            zr.token_logprobs(first, ids, ref)
            for _ in range(2):
                z = net.forward(x)
                zr.policy_loss(z, ids, old, advantage, out, grad=z, weight=weight, ref_logp=ref, kl=0.02, logp=logp, plan=net.plan)
                net.backward(z)
                rep = net.step(hyper)
            history.append(float(reward.mean()))
        if step % 10 == 0 or step == steps - 1:
            report(f"step {step:3d}  {'loss' if loss == 'preference' else 'reward'} {history[-1]:.4f}  scale {rep.scale:.0f}{'  skipped' if rep.skipped else ''}")
    zr.mx4_status()
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("policy", "preference"), default="policy")
    for name, value in (("tokens", 1024), ("dim", 256), ("hidden", 512), ("vocab", 2000), ("steps", 30)):
        ap.add_argument(f"--{name}", type=int, default=value)
    train(**vars(ap.parse_args()))
