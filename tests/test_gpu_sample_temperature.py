"""Temperatures at which the distance between two logits does not fit FP32 and still weighs
something, and those beyond FP32's range."""
import pytest
import torch

from test_gpu_sample import check, rows, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1e30, 6e37, 1e38, 3e38, 1e39, 1e60, 1e300])
def test_logits_as_large_as_the_type_holds(dtype, T):
    # -3e38 to 3e38: a distance of up to 6e38
    x, u = 3e38 * (2 * torch.rand(12, 1001, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) - 1), \
        uniforms(12, 4)
    x = x.to(rows(1, 1, dtype, 0).dtype)
    assert torch.isfinite(x.float()).all()
    for kw in (dict(), dict(top_k=300), dict(top_p=0.6), dict(min_p=0.3)):
        check(x, u, temperature=T, **kw)
    if T < 1e39:
        check(x, u, temperature=torch.full((12,), T, device="cuda"))
