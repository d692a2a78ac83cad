"""The divergence of the policy loss: watched without a weight, and its accuracy.

Bounds of k = exp(d) - d - 1 (e = 2^-24) for d that FP32 holds:
  |d| < 1   d^2 times a polynomial of ten terms c_j = 1 / (j + 2)!: Horner's rule
            is off by e sum (2 j + 1) c_j |d|^j, the coefficients by e sum c_j |d|^j,
            together at most 5.5 e of the polynomial (at d = -1); e each for the two
            products, and less than 2^-27 for the terms left out: 8 e k
  else      exp(d), of at most two steps (4 e), then a rounding of each difference:
            e (4 exp(d) + |exp(d) - d| + k)
"""
import math

import numpy as np
import pytest
import torch

from gpu_util import bits_equal

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def exact(d):
    """exp(d) - d - 1 in 64 bits, by its series where the difference cancels."""
    if abs(d) < 0.1:
        return math.fsum(d ** j / math.factorial(j) for j in range(2, 14))
    return math.expm1(d) - d


def test_divergence_of_single_tokens(lib):
    rng = np.random.default_rng(1)
    ds = np.concatenate([
        rng.uniform(-1, 1, 150), rng.uniform(-4, 4, 60), 10.0 ** rng.uniform(-8, 0, 40),
        -(10.0 ** rng.uniform(-8, 0, 40)), [1.0, -1.0, np.nextafter(np.float32(1), np.float32(0)),
                                            np.nextafter(np.float32(-1), np.float32(0)), 20.0, -50.0]])
    ref = torch.tensor(ds, dtype=torch.float32, device="cuda")
    zero = torch.zeros_like(ref)
    got = [lib.policy_loss(zero[i:i + 1], zero[i:i + 1], zero[i:i + 1], ref_logp=ref[i:i + 1])[0]
           for i in range(len(ds))]
    for d, g in zip(ref.tolist(), torch.stack(got)[:, 2].tolist()):
        k = exact(d)
        b = 8 * E * k if abs(d) < 1 else E * (4 * math.exp(d) + abs(math.exp(d) - d) + k)
        assert abs(g - k) <= b + 2.0 ** -149, d


@pytest.mark.parametrize("N", [3, 4096, 20011])
@pytest.mark.parametrize("seqs", [False, True])
@pytest.mark.parametrize("bad", [90.0, float("inf"), float("nan")])
def test_a_watched_divergence_that_overflows(lib, N, seqs, bad):
    """kl_coef = 0: the divergence is no part of the loss, whatever it is."""
    g = torch.Generator(device="cuda").manual_seed(N)
    logp = -torch.rand(N, device="cuda", generator=g)
    old, adv = logp + 0.1, torch.randn(N, device="cuda", generator=g)
    ref = logp.clone()
    ref[N // 2] += bad
    offs = torch.tensor([0, N // 3, N // 3, N], device="cuda") if seqs else None
    stats, grad = lib.policy_loss(logp, old, adv, ref_logp=ref, seq_offsets=offs)
    plain, plain_grad = lib.policy_loss(logp, old, adv, seq_offsets=offs)
    assert not math.isfinite(float(stats[2])) and math.isfinite(float(stats[0]))
    assert bits_equal(stats[:2].contiguous(), plain[:2].contiguous())
    assert bits_equal(stats[3:].contiguous(), plain[3:].contiguous()) and bits_equal(grad, plain_grad)
    assert float(stats[0]) == float(stats[1])
    with_it, _ = lib.policy_loss(logp, old, adv, ref_logp=ref, seq_offsets=offs, kl_coef=0.1)
    assert not math.isfinite(float(with_it[0]))
