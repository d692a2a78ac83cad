"""A min_p that leaves many tokens of rows whose logits share a large offset: the tokens that
the sums hold and those that the draw goes through are the same ones.  Where no token lies next
to min_p's border, that is by the exponents x log2(e) / T - ref, which an offset leaves alone."""
import pytest
import torch

import cross_entropy_rl_gb300 as ll
from test_gpu_sample import check, rows, uniforms

pytestmark = pytest.mark.gpu
V = 70001  # 274 groups of 256 logits: more than the 256 whose tokens go to a list


def drawn(x, u, **kw):
    """check(), with outputs that a draw has to overwrite."""
    N = x.shape[0]
    out = (torch.full((N,), -7, dtype=torch.int64, device="cuda"),
           torch.full((N,), 7.0, device="cuda"), torch.full((N,), 7.0, device="cuda"))
    tokens = check(x, u, out=out, **kw)
    assert (tokens >= 0).all() and (out[1] <= 0).all() and (out[2] <= 0).all()


# rows in clusters, and a block each with a second launch in clusters
@pytest.mark.parametrize("N", [40, 120])
@pytest.mark.parametrize("offset", [0.0, 3000.0, -20000.0, 20000.0, 1e5, -1e5])
def test_wide_min_p(N, offset):
    for i, min_p in enumerate((0.00113, 0.00171, 0.00237, 0.00331)):
        x = rows(N, V, "f32", 100 + i) + offset
        drawn(x, uniforms(N, 200 + i), min_p=min_p)


@pytest.mark.parametrize("dtype,offset,T", [("f32", 300.0, 0.01), ("f32", -5000.0, 0.5),
                                            ("bf16", 2000.0, 6.0), ("f16", -3000.0, 2.0)])
def test_wide_min_p_at_a_temperature(dtype, offset, T):
    x = (T * rows(60, V, "f32", 300) + offset).to(rows(1, 1, dtype, 0).dtype)
    for i, min_p in enumerate((0.00119, 0.0023)):
        drawn(x, uniforms(60, 301 + i), min_p=min_p, temperature=T)


def test_wide_min_p_and_top_p():
    x, u = rows(60, V, "f32", 310) + 50000.0, uniforms(60, 311)
    drawn(x, u, min_p=0.0017, top_p=0.999)
    drawn(x, u, min_p=0.0017, top_p=0.5)
    same = ll.sample(x[:30], u[:30], min_p=0.0017)  # in clusters and by blocks: the same bits
    assert all(torch.equal(a, b[:30]) for a, b in zip(same, ll.sample(x, u, min_p=0.0017)))
