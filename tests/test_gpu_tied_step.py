"""The training step of examples/tied_policy_step.py: its gradients against
automatic differentiation of the same model in 64 bits, and that it learns."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tied_policy_step.py")


@pytest.fixture(scope="module")
def example(lib):
    spec = importlib.util.spec_from_file_location("tied_policy_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def loss64(W, A, B, scale, context, answer, old, adv, mask, offs, beta, lo=0.2, hi=0.2):
    e = W[context] * scale
    h = e + torch.tanh(e @ A) @ B
    logp = torch.log_softmax(h @ W.t(), 1)[torch.arange(len(answer)), answer.clamp_min(0)]
    r = (logp - old).exp()
    p = -torch.minimum(r * adv, r.clamp(1 - lo, 1 + hi) * adv)
    d = old - logp
    k = d.exp() - d - 1
    total, full = 0.0, 0
    for b in range(len(offs) - 1):
        m = mask[offs[b]:offs[b + 1]]
        if m.any():
            full += 1
            total = total + (p + beta * k)[offs[b]:offs[b + 1]][m].mean()
    return total / full


def test_gradients(example):
    """FP32 operands.  The contractions are within 5e-4 of themselves (the FP32
    tolerance of every gradient of the library); the table's adds three of them, the
    others two: 2e-3 of the largest entry holds them all."""
    V, D, N = 96, 64, 700
    m = example.Model(V, D, torch.float32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    context = torch.randint(0, V, (N,), device="cuda", generator=g)
    answer = torch.randint(0, V, (N,), device="cuda", generator=g)
    mask = torch.rand(N, device="cuda", generator=g) > 0.3
    answer = torch.where(mask, answer, -100)
    old = m.sample(context, g)[1] * 0
    with torch.no_grad():
        h = m.hidden(context)[2]
        z = torch.log_softmax((h @ m.W.t()).double(), 1)
        old = z[torch.arange(N), answer.clamp_min(0)].float()
        old += 0.15 * torch.randn(N, device="cuda", generator=g)
    adv = torch.randn(N, device="cuda", generator=g)
    offs = [0, 0, 50, 51, 400, 700]
    _, grads = m.loss_and_grads(context, answer, old, adv, ref_logp=old, mask=mask, kl_coef=0.2,
                                seq_offsets=torch.tensor(offs, device="cuda"))
    p = [x.double().cpu().requires_grad_() for x in m.master]
    c = [x.cpu() for x in (context, answer, old.double(), adv.double(), mask)]
    loss64(*p, m.scale, *c, offs, 0.2).backward()
    for got, ref in zip(grads, p):
        err = np.abs(got.double().cpu().numpy() - ref.grad.numpy()).max()
        assert err <= 2e-3 * float(ref.grad.abs().max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_it_learns(example, dtype):
    r = example.train(400, dtype=dtype, log=lambda s: None)
    assert np.mean(r[-10:]) > 10 * np.mean(r[:10]) and np.mean(r[-10:]) > 0.3
