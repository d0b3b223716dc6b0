"""The example that runs the layers, the losses and the ZeRO step together: it runs, and its gradients are those of the
network that its 4-bit operands stand for, each in 64 bits."""
import importlib.util
import math
import os

import pytest
import torch

import zero_gradient_reduction_gb300 as zr

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("policy_mx4", os.path.join(ROOT, "examples", "policy_mx4.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("loss", ["policy", "preference"])
def test_example_runs(example, loss):
    history = example.train(loss=loss, tokens=200, dim=96, hidden=160, vocab=301, steps=4, report=lambda _: None)
    assert len(history) == 4 and all(math.isfinite(h) for h in history)


def test_the_same_seed_gives_the_same_run(example):
    runs = [example.train(loss="preference", tokens=100, dim=64, hidden=96, vocab=130, steps=3, report=lambda _: None) for _ in range(2)]
    assert runs[0] == runs[1]


def values(q):
    out = torch.empty(q.rows, q.cols, device="cuda")
    zr.mx4_dequantize(q, out)
    return out.double()


def close(got, want, steps, what):
    """Sums of a few hundred fp32 products, then `steps` half units of bf16 of the largest value."""
    tol = (1e-5 + steps * 2.0 ** -8) * float(want.abs().max())
    assert float((got.double() - want).abs().max()) <= tol, what


def test_forward_and_backward(example):
    """Every product and sum of a pass against 64 bits from the 4-bit operands that the pass holds; the loss's gradient
    against autograd through a log softmax."""
    T, D, F, V = 96, 64, 80, 130
    g = torch.Generator(device="cuda").manual_seed(3)
    net = example.Network(T, D, F, V, g)
    net.master("b1").normal_(0, 0.5, generator=g)
    net.master("b2").normal_(0, 0.5, generator=g)
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    z = net.forward(x)
    pre = values(net.x4[0]) @ values(net.w1[0]).t() + net.master("b1").double()
    close(net.pre, pre, 1, "pre")
    close(net.h, torch.nn.functional.gelu(pre, approximate="tanh"), 1, "h")
    close(net.y, values(net.h4[0]) @ values(net.w2[0]).t() + net.master("b2").double() + x.double(), 1, "y")
    close(z, values(net.y4[0]) @ values(net.e[0]).t(), 1, "logits")

    ids, old = torch.randint(0, V, (T,), generator=g, device="cuda"), torch.empty(T, device="cuda")
    advantage, loss = torch.randn(T, generator=g, device="cuda"), torch.empty(T, device="cuda")
    zr.token_logprobs(z, ids, old)
    zs = z.double().requires_grad_()
    logp = torch.log_softmax(zs, 1).gather(1, ids[:, None])[:, 0]
    ratio = torch.exp(logp - logp.detach() + 0.05)
    old -= 0.05
    want = -torch.minimum(ratio * advantage, ratio.clamp(0.8, 1.2) * advantage)
    want.sum().backward()
    zr.policy_loss(z, ids, old, advantage, loss, grad=z, plan=net.plan)
    close(loss, want.detach(), 0, "loss")
    close(z, zs.grad * 1024.0, 1, "the loss's gradient")

    net.backward(z)
    close(net.dy, values(net.dz4[0]) @ values(net.e[1]).t(), 1, "dY")
    close(net.grad("e"), values(net.dz4[1]) @ values(net.y4[1]).t(), 0, "dE")
    close(net.grad("b2"), net.dy.double().sum(0), 0, "db2")
    close(net.grad("w2"), values(net.dy4[1]) @ values(net.h4[1]).t(), 0, "dW2")
    p = net.pre.double().requires_grad_()
    torch.nn.functional.gelu(p, approximate="tanh").backward(values(net.dy4[0]) @ values(net.w2[1]).t())
    close(net.dh, p.grad, 1, "dH")
    close(net.grad("b1"), net.dh.double().sum(0), 0, "db1")
    close(net.grad("w1"), values(net.dh4[1]) @ values(net.x4[1]).t(), 0, "dW1")
