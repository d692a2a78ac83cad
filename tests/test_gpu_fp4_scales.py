"""Products of 4-bit matrices whose two FP32 scales have a product outside FP32's normal range."""
import pytest
import torch

import cross_entropy_rl_gb300 as ll
from rollout_util import quantize, values
from test_gpu_fp4 import HALF, TINY

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [5, 200])  # both kernels of the product
@pytest.mark.parametrize("gh,gw,size", [
    (1e-21, 1e-21, 2000.0), (1e-23, 1e-23, 2000.0), (1e-22, 3e-25, 2000.0), (1e-38, 1e-38, 2000.0),
    (1e-44, 1e-3, 2000.0), (1e20, 1e20, 0.02), (3e21, 1e17, 0.5), (1e30, 1e-30, 1.0), (1e38, 1e-38, 3.0)])
def test_scales_far_from_1(out, N, gh, gw, size):
    g = torch.Generator(device="cuda").manual_seed(N)
    K, V = 320, 259
    scale = [torch.tensor(s, device="cuda") for s in (gh, gw)]
    # values up to about `size` scales (2688 is the largest that the format holds), FP32 subnormals
    # among them where the scale is close to those
    x = [(torch.randn(r, K, device="cuda", generator=g).double() * size / 4 * s.double()).float()
         for r, s in zip((N, V), scale)]
    x[0][3] = 0.0
    q = [ll.fp4_quantize(t, "nv", scale=s) for t, s in zip(x, scale)]
    v = []
    for t, s in zip(x, scale):
        v.append(torch.from_numpy(values(*quantize(t.cpu().numpy(), "nv", s.cpu().numpy())[:2], "nv",
                                         float(s))).cuda())
    top = float(torch.finfo(out).max)
    for b in (None, 3e-36 * torch.randn(V, device="cuda", generator=g)):
        got = ll.fp4_linear(*q, b, out_dtype=out).double()
        want, whole = v[0] @ v[1].T, v[0].abs() @ v[1].abs().T
        if b is not None:
            want, whole = want + b.double(), whole + b.double().abs()
        # as for scales near 1: an FP32 sum that the tensor cores may truncate at each 64 products,
        # two products with the scales, the bias, the rounding to `out`; 2^-149 for each rounding of
        # a subnormal number on the way
        tol = whole * (K / 64 + 10) * 2.0 ** -22 + want.abs() * HALF[out] + TINY[out] + 3 * 2.0 ** -149
        near = want.abs() * (1 + 2.0 ** -7) + tol < top
        assert not torch.isnan(got).any()
        assert ((got - want).abs() <= tol)[near].all()
        if b is None:
            assert (got[3] == 0).all()
