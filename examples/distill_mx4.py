"""Training an output layer in 4 bits from a teacher's top logits, with the 4-bit operators and the ZeRO step together.

A student's fp32 masters W live in a plan's state. Each step quantises them and the hidden states X to microscaled
4-bit floating point, multiplies (logits = X W^T), takes the distillation loss against the teacher's top logits with
its gradient times the plan's loss scale in place of the logits, quantises that gradient by chance and multiplies
twice: dX = dY W for the layers below, and dW = dY^T X straight into the gradient replica that the step reduces.
A gradient that overflows makes the step skip and halve the scale, which the next loss reads on the device.

    python examples/distill_mx4.py [--tokens 2048 --dim 512 --vocab 4000 --top 32 --steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_gradient_reduction_gb300 as zr  # noqa: E402


def train(tokens=2048, dim=512, vocab=4000, top=32, steps=60, temperature=2.0, seed=0, report=print):
    """Mean loss of each step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, dim, generator=g, device="cuda").bfloat16()
    teacher_w = 0.2 * torch.randn(vocab, dim, generator=g, device="cuda")
    teacher, ids = torch.topk(x.float() @ teacher_w.t(), top)  # what a teacher's pass over the tokens keeps
    weight = torch.full((tokens,), 1.0 / tokens, device="cuda")

    plan = zr.Plan([vocab * dim], W=1, dtype=zr.BF16, stage=1, cap=vocab * dim, fp32_grads=True,
                   scaler=zr.Scaler(init_scale=65536.0, dynamic=True))
    state, hyper = plan.new_state(), zr.AdamW(lr=3e-3, weight_decay=0.0)
    state.master[0].normal_(0, 0.02, generator=g)
    zr.all_gather(state.master[0], [state.param[0]])
    grads = [torch.zeros(plan.numel, device="cuda")]
    dw = grads[0][:vocab * dim].view(vocab, dim)

    xq, x_t = zr.Mx4(tokens, dim), zr.Mx4(dim, tokens)
    w, w_t = zr.Mx4(vocab, dim), zr.Mx4(dim, vocab)
    dy, dy_t = zr.Mx4(tokens, vocab), zr.Mx4(vocab, tokens)
    logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    loss = torch.empty(tokens, device="cuda")
    rand = torch.empty(tokens, vocab, dtype=torch.uint8, device="cuda")

    zr.mx4_quantize(x, xq, x_t)
    live, losses = 0, []
    for step in range(steps):
        zr.mx4_quantize(state.live(live)["master"][:vocab * dim].view(vocab, dim), w, w_t)
        zr.mx4_matmul(xq, w, logits)
        zr.distill_topk(logits, ids, teacher, loss, grad=logits, weight=weight, temperature=temperature, plan=plan)
        rand.random_(0, 256, generator=g)
        zr.mx4_quantize(logits, dy, dy_t, rand=rand)
        zr.mx4_matmul(dy, w_t, dx)
        zr.mx4_matmul(dy_t, x_t, dw)
        rep = plan.step(grads, state, hyper, report=True)
        live = rep.current
        losses.append(float(loss.sum()))
        if step % 10 == 0 or step == steps - 1:
            report(f"step {step:3d}  loss {losses[-1]:.4f}  scale {rep.scale:.0f}{'  skipped' if rep.skipped else ''}")
    zr.mx4_status()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("dim", 512), ("vocab", 4000), ("top", 32), ("steps", 60)):
        ap.add_argument(f"--{name}", type=int, default=value)
    train(**vars(ap.parse_args()))
