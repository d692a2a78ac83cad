"""The embedding gradient next to the sizes at which its path changes: 1024 tokens
(matching or a sort), 2048 (one block or a cluster), 32768 (a cluster or the device).
Small whole numbers, whose sums are exact in any order, and the bits of random ones."""
import numpy as np
import pytest
import torch

from gpu_util import bits_equal, host64

pytestmark = pytest.mark.gpu

SIZES = [1023, 1024, 1025, 1500, 2047, 2048, 2049]


def ids(N, V, seed, hot, invalid):
    rng = np.random.default_rng(seed)
    y = rng.integers(0, V, N)
    y[rng.random(N) < hot] = V // 2
    near = rng.random(N) < 0.3  # tokens side by side in the table too
    y = np.where(near, np.minimum(y % 300, V - 1), y)
    return np.where(rng.random(N) < invalid, rng.choice([-100, -1, V, 2 ** 40], N), y)


@pytest.mark.parametrize("N", SIZES)
@pytest.mark.parametrize("V,D,invalid", [
    (1, 8, 0.0), (2, 40, 0.97), (511, 264, 0.97), (513, 8, 0.0), (9000, 515, 0.05), (300000, 8, 0.05),
    (140000000, 1, 0.97)])
def test_sums(lib, N, V, D, invalid):
    rng = np.random.default_rng(N + V)
    y = ids(N, V, N, 0.1, invalid)
    g = torch.from_numpy(rng.integers(-3, 4, (N, D))).to(torch.bfloat16).cuda()
    ok = (y >= 0) & (y < V)
    rows, back = np.unique(y[ok], return_inverse=True)
    want = np.zeros((len(rows), D))
    np.add.at(want, back, host64(g)[ok])
    at, yc = torch.from_numpy(rows).cuda(), torch.from_numpy(y).cuda()
    got = torch.full((V, D), float("nan"), device="cuda")
    lib.embed_backward(g, yc, V, scale=2.0, out=got)
    assert (host64(got[at]) == 2 * want).all()
    got[at] = 0
    assert float(got.abs().max()) == 0
    lib.embed_backward(g, yc, V, accumulate=True, out=got.fill_(1))
    assert (host64(got[at]) == 1 + want).all()
    got[at] = 1
    assert float(got.min()) == 1 == float(got.max())
    del got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [1024, 1500, 2048, 2049])
@pytest.mark.parametrize("hot", [0.0, 0.7])
def test_bits_and_rows(lib, N, hot):
    """The same bits from run to run, from shards of the vocabulary, and for a
    token whatever the other tokens are."""
    V, D = 3000, 72
    g = torch.randn(N, D, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
    y = ids(N, V, N, hot, 0.05)
    yc = torch.from_numpy(y).cuda()
    a = lib.embed_backward(g, yc, V)
    assert bits_equal(a, lib.embed_backward(g, yc, V))
    assert bits_equal(a, lib.embed_backward(g, yc, V, accumulate=True, out=torch.zeros_like(a)))
    for lo, hi in ((0, 1000), (1000, 1513), (1513, 3000)):
        assert bits_equal(a[lo:hi].contiguous(), lib.embed_backward(g, yc, hi - lo, v0=lo))
    for v in (V // 2, int(y[(y >= 0) & (y < V)][0])):
        other = np.where(y == v, y, (y * 7 + 1) % V)
        other = np.where((other == v) & (y != v), -100, other)
        b = lib.embed_backward(g, torch.from_numpy(other).cuda(), V)
        assert bits_equal(a[v].contiguous(), b[v].contiguous())


@pytest.mark.parametrize("N", [1500, 2048])
def test_graph(lib, N):
    """A captured call of one sorting block, replayed on other tokens."""
    V, D = 5000, 24
    g = torch.randn(N, D, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16).cuda()
    y = torch.from_numpy(ids(N, V, 52, 0.3, 0.1)).cuda()
    dW, dA = torch.empty(V, D, device="cuda"), torch.zeros(V, D, device="cuda")
    ws = torch.empty(lib.load().ll_embed_workspace_size(N, D, V), dtype=torch.uint8, device="cuda")
    lib.embed_backward(g, y, V, out=dW, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.embed_backward(g, y, V, out=dW, workspace=ws)
        lib.embed_backward(g, y, V, out=dA, workspace=ws, accumulate=True)
    y.copy_(torch.from_numpy(ids(N, V, 53, 0.6, 0.3)).cuda())
    ws.random_(0, 256)  # a replay may find anything in its workspace
    dA.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = lib.embed_backward(g, y, V)
    assert bits_equal(dW, want) and bits_equal(dA, want)
