"""Rows whose tokens above the floor do not fit the list: its length, which every thread has
read by then, is cleared for the next list only after that.  Many calls, each with the bits
of the first; rows in clusters, and a block each with a second launch in clusters."""
import pytest
import torch

import cross_entropy_rl_gb300 as ll
from test_gpu_sample import check, rows, uniforms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [40, 2100])
@pytest.mark.parametrize("kw", [dict(min_p=0.01), dict(top_p=0.9), dict(min_p=0.003, top_p=0.9)], ids=str)
def test_lists_that_overflow(dtype, N, kw):
    x, u = rows(N, 6001, dtype, 81, scale=0.1), uniforms(N, 82)
    check(x[:50], u[:50], **kw)
    want = ll.sample(x, u, **kw)
    for _ in range(200):
        got = ll.sample(x, u, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ll.check_status() == 0
