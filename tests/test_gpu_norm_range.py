"""The gradient norm where squares and their sums come near the end of the FP32 range.

Bounds (e = 2^-24): the squares are FP32 sums of at most 32 terms, each with one
rounding: 32 e of a sum at the most, 16 e of its root; what is added to pairs of
FP32 values from there on (each to about 2^-44 of itself, a few thousand of them
one after another) stays below e; e for the result's rounding: 18 e.  An element
after clipping: that, e each for the bound and 1e-6 as FP32 values, the sum, the
division and the product, and the half step of its type."""
import math

import pytest
import torch

from gpu_util import bits_equal

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
STEP = {torch.float32: E, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
NORM = 18 * E


@pytest.mark.parametrize("n,value,dt", [
    (1 << 27, 2.0 ** 55, torch.float32), (1 << 27, 2.0 ** 50, torch.float32),
    (1 << 27, 2.0 ** 38, torch.float32), (1 << 27, 1.5 * 2.0 ** 38, torch.float32),
    (500000000, 2e16, torch.bfloat16), ((1 << 27) + 5, 2.0 ** -50, torch.float32),
    ((1 << 27) + 5, 2.0 ** -51, torch.float32), (3000, 2.0 ** 55, torch.float32)])
def test_many_elements_of_one_size(lib, n, value, dt):
    t = torch.full((n,), value, dtype=dt, device="cuda")
    value = float(t[0])
    want = value * math.sqrt(n)
    assert abs(float(lib.grad_norm([t])) - want) <= NORM * want
    bound = want / 1024
    norm = lib.clip_grads([t], bound)
    assert abs(float(norm) - want) <= NORM * want
    coef = bound / (want + 1e-6)
    low, high = (float(x) for x in t.aminmax())
    assert low == high
    assert abs(low - value * coef) <= (NORM + 5 * E + STEP[dt] * (1 + 32 * E)) * value * coef
    del t
    torch.cuda.empty_cache()


def test_many_launches_of_large_sums(lib):
    """More than a thousand launches whose blocks' sums come near 2^110."""
    x = torch.full((4096,), math.sqrt(0.5) * 2.0 ** 49, device="cuda")
    value, count = float(x[0]), 600000
    want = value * math.sqrt(4096 * count)
    assert abs(float(lib.grad_norm([x] * count)) - want) <= NORM * want


@pytest.mark.parametrize("sizes", [[(1000,), (7,)], [(3000001,), (513, 700), (5,)]])
@pytest.mark.parametrize("scale", [1e-16, 2.0 ** -50, 1e-3, 2.0 ** 38, 1e12, 1e15, 1e17, 3e20])
def test_norm_of_random_elements(lib, sizes, scale):
    """Runs on both sides of the borders of what is squared in 32 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    ts = [torch.randn(s, device="cuda", generator=g) * scale for s in sizes]
    want = math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))
    assert abs(float(lib.grad_norm(ts)) - want) <= NORM * want


@pytest.mark.parametrize("n", [2000, 700001])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("given", [False, True])
def test_an_infinite_bound_writes_nothing(lib, n, bad, given):
    """max_norm = infinity: no clipping, whatever the norm."""
    ts = [torch.randn(n, device="cuda"), torch.randn(33, device="cuda").bfloat16()]
    ts[0][n // 2] = bad
    keep = [t.clone() for t in ts]
    norm = lib.clip_grads(ts, float("inf"), norm=lib.grad_norm(ts) if given else None)
    assert math.isnan(bad) and math.isnan(float(norm)) or float(norm) == float("inf")
    assert all(bits_equal(a, b) for a, b in zip(ts, keep))
