"""Lists of tokens that are full to the last place while further tokens wait."""
import pytest
import torch

from test_gpu_sample import TORCH, check, rows, uniforms

pytestmark = pytest.mark.gpu


# rows in clusters, and a block each
@pytest.mark.parametrize("N", [40, 120])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("more", [0, 1, 300])
def test_1024_tokens_and_more(N, dtype, more):
    # a grammar leaves 1024 tokens of the first five groups of 256 (of the last one's lanes none
    # is reached), and `more` of the sixth and seventh, all in one range of groups
    V = 151936
    keep = torch.zeros(V, dtype=torch.bool, device="cuda")
    for g in range(4):
        keep[256 * g:256 * g + 248] = True
    keep[1024:1024 + 32] = True
    keep[1280:1280 + more] = True
    assert int(keep.sum()) == 1024 + more
    x = torch.full((N, V), float("-inf"), device="cuda", dtype=TORCH[dtype])
    x[:, keep] = rows(N, 1024 + more, dtype, more, scale=0.5)
    if more == 1:
        x[:, 1280] = 6.0
    for kw in (dict(min_p=1e-4), dict(top_p=0.9999), dict(top_p=0.99, min_p=1e-5)):
        check(x, uniforms(N, 7), **kw)
