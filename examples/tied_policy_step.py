"""A policy trained with the library's calls from tokens to clipped gradients.

The model is one block between a vocabulary table that is tied: its rows embed
the context tokens and score the answer tokens.

    e = embed(W, context)                      ll.embed_forward
    h = e + tanh(e A) B                        (torch)
    logp = log softmax(h W^T)[answer]          ll.forward
    loss, grad_logp = policy loss              ll.policy_loss
    grad_h, grad_W = ...                       ll.backward
    grad_e, grad_A, grad_B = ...               (torch)
    grad_W += embedding's                      ll.embed_backward(accumulate=True)
    all gradients clipped as one vector        ll.clip_grads

The task: the answer to context token c is (7 c + 3) mod V; answers are sampled
and rewarded, several updates are made on each batch of them.

    python examples/tied_policy_step.py [--updates N] [--dtype bf16|f32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import cross_entropy_rl_gb300 as ll  # noqa: E402


class Model:
    """FP32 master weights; the products run on copies of `dtype`."""

    def __init__(self, V, D, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.scale = dtype, D ** 0.5
        self.master = [torch.randn(s, device="cuda", generator=g) * D ** -0.5
                       for s in ((V, D), (D, D), (D, D))]
        self.cast()

    def cast(self):
        self.W, self.A, self.B = (p.to(self.dtype) for p in self.master)

    def hidden(self, context):
        e = ll.embed_forward(self.W, context, scale=self.scale)
        t = torch.tanh(e @ self.A)
        return e, t, e + t @ self.B

    def sample(self, context, g):
        """Answers of the policy and their logp."""
        h = self.hidden(context)[2]
        y = torch.softmax((h @ self.W.t()).float(), 1).multinomial(1, generator=g)[:, 0]
        return y, ll.forward(h, self.W, None, y)[0]

    def loss_and_grads(self, context, answer, old_logp, advantages, **loss):
        """(stats, [grad_W, grad_A, grad_B] in FP32)."""
        e, t, h = self.hidden(context)
        logp, lse = ll.forward(h, self.W, None, answer)
        stats, grad_logp = ll.policy_loss(logp, old_logp, advantages, **loss)
        gh, gW, _ = ll.backward(grad_logp, h, self.W, None, answer, lse)
        u = (gh @ self.B.t()) * (1 - t * t)
        ge = gh + u @ self.A.t()
        ll.embed_backward(ge, context, self.W.shape[0], scale=self.scale, accumulate=True, out=gW)
        return stats, [gW, (e.t() @ u).float(), (t.t() @ gh).float()]

    def update(self, grads, lr, max_norm):
        norm = ll.clip_grads(grads, max_norm)
        for p, g in zip(self.master, grads):
            p.sub_(g, alpha=lr)
        self.cast()
        return norm


def train(updates=200, V=64, D=64, dtype=torch.bfloat16, seqs=48, lr=1.0, seed=0, log=print):
    """Mean reward of each batch of answers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    model, rewards = Model(V, D, dtype, seed), []
    for batch in range(updates // 4):
        # ragged sequences; the last token of some is padding
        lengths = torch.randint(1, 60, (seqs,), device="cuda", generator=g)
        offsets = torch.cat([lengths.new_zeros(1), lengths.cumsum(0)])
        N = int(offsets[-1])
        context = torch.randint(0, V, (N,), device="cuda", generator=g)
        answer, old = model.sample(context, g)
        mask = torch.rand(N, device="cuda", generator=g) > 0.05
        answer = torch.where(mask, answer, -100)
        reward = (answer == (7 * context + 3) % V).float()
        rewards.append(float(reward[mask].mean()))
        adv = (reward - rewards[-1]) / max((rewards[-1] * (1 - rewards[-1])) ** 0.5, 1e-2)
        for _ in range(4):
            stats, grads = model.loss_and_grads(context, answer, old, adv, ref_logp=old, mask=mask,
                                                seq_offsets=offsets, kl_coef=0.01, clip_high=0.28)
            norm = model.update(grads, lr, 1.0)
        if batch % 10 == 0:
            log("batch %3d  reward %.3f  loss %+.4f  divergence %.4f  clipped %.3f  norm %.3f" % (
                batch, rewards[-1], stats[0], stats[2], stats[3], norm))
    assert ll.check_status() == 0
    return rewards


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--updates", type=int, default=800)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    r = train(a.updates, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    print("mean reward of the first and last ten batches: %.3f, %.3f" % (
        sum(r[:10]) / 10, sum(r[-10:]) / 10))
