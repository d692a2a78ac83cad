"""Embedding lookup and its gradient against their definitions in 64 bits.

Bounds, with u the half step of the output type (2^-8 bf16, 2^-11 fp16, 2^-24
fp32) and an FP32 half step of 2^-24:
  lookup    the product is rounded to FP32 and then to the output:
            |err| <= (u + 2^-24) |r|  (+ half the smallest step of fp16)
  gradient  c terms, the scaling and the table's entry: at most c + 3 roundings
            of values no larger than M = |table| + |scale| sum |g|, then the
            output's: |err| <= (c + 3) 2^-24 M + u (|r| + (c + 3) 2^-24 M)
"""
import numpy as np
import pytest
import torch

from gpu_util import TORCH, assert_pos_zero, bits_equal, host64

pytestmark = pytest.mark.gpu

STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


def table(rows, cols, dt, seed, pad=0, shift=0):
    """[rows, cols] normal values in a buffer `pad` columns wider that starts
    `shift` elements into its allocation."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(rows * (cols + pad) + shift, generator=g).to(TORCH[dt]).cuda()
    return buf[shift:].view(rows, cols + pad)[:, :cols]


def ids(N, V, seed, hot=0.0, invalid=0.0, v0=0):
    rng = np.random.default_rng(seed)
    y = rng.integers(0, V, N)
    y[rng.random(N) < hot] = V // 2
    y = y + v0
    bad = rng.random(N) < invalid
    y[bad] = rng.choice([-100, v0 - 1, v0 + V, 2**40, -2**40, 2**63 - 1, -2**63], bad.sum())
    return y


# ---------------------------------------------------------------------- lookup
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                    ("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"),
                                    ("f16", "f32")])
@pytest.mark.parametrize("N,D,V,pad,shift", [
    (1, 1, 1, 0, 0), (1, 4096, 100, 0, 0), (7, 8, 5, 0, 0), (33, 515, 64, 0, 0),
    (64, 136, 999, 8, 0), (9, 1031, 50, 3, 1), (300, 72, 4099, 0, 8), (5, 9000, 11, 24, 0)])
def test_lookup(lib, dt, out, N, D, V, pad, shift):
    W = table(V, D, dt, 1, pad, shift)
    y = ids(N, V, 2, invalid=0.2)
    scale = 3.7
    got = lib.embed_forward(W, torch.from_numpy(y).cuda(), scale=scale, out_dtype=TORCH[out])
    assert got.dtype == TORCH[out] and got.shape == (N, D)
    ok = (y >= 0) & (y < V)
    ref = np.where(ok[:, None], host64(W)[np.where(ok, y, 0)] * np.float64(np.float32(scale)), 0.0)
    err = np.abs(host64(got) - ref)
    assert (err <= (STEP[out] + 2.0 ** -24) * np.abs(ref) + TINY[out]).all()
    if (~ok).any():
        assert_pos_zero("rows of other tokens", got[torch.from_numpy(~ok).cuda()])


def test_lookup_leaves_the_rest_of_a_row(lib):
    W = table(40, 24, "bf16", 3)
    y = torch.from_numpy(ids(17, 40, 4)).cuda()
    for D, ld, shift in ((24, 40, 0), (24, 27, 0), (24, 32, 1)):
        buf = torch.full((17 * ld + shift,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[shift:].view(17, ld)
        lib.embed_forward(W, y, out=out[:, :D])
        assert bits_equal(out[:, :D].contiguous(), W[y])
        assert (out[:, D:] == 7).all() and (buf[:shift] == 7).all()


def test_lookup_shards_add_up(lib):
    W = table(1000, 64, "bf16", 5)
    y = torch.from_numpy(ids(400, 1000, 6, invalid=0.1)).cuda()
    whole = lib.embed_forward(W, y, scale=8.0)
    parts = [lib.embed_forward(W[a:b], y, scale=8.0, v0=a) for a, b in ((0, 300), (300, 301), (301, 1000))]
    assert bits_equal(parts[0] + parts[1] + parts[2], whole)
    assert sum((p != 0).any(1).int() for p in parts).max() <= 1


def test_lookup_keeps_special_values(lib):
    W = torch.tensor([[float("inf"), -float("inf"), float("nan"), 65504.0, 1e-7, -0.0, 0.0, 1.0]],
                     dtype=torch.float16, device="cuda")
    y = torch.tensor([0, 1, 0], device="cuda")
    got = lib.embed_forward(W, y, scale=2.0).float().cpu()
    ref = (W.float() * 2).half().float().cpu()[0]
    for n in (0, 2):
        assert torch.equal(got[n].nan_to_num(9), ref.nan_to_num(9))
    assert_pos_zero("other token", got[1])


# -------------------------------------------------------------------- gradient
def reference(g, y, V, scale, start, v0=0):
    """(sum, M, c) of the definition: FP64 sums, the magnitudes they add, and the
    number of terms of each row."""
    g = host64(g)
    y = y - v0
    ok = (y >= 0) & (y < V)
    r, M = np.zeros((V, g.shape[1])), np.zeros((V, g.shape[1]))
    s = np.float64(np.float32(scale))
    np.add.at(r, y[ok], g[ok] * s)
    np.add.at(M, y[ok], np.abs(g[ok] * s))
    c = np.bincount(y[ok].astype(np.int64), minlength=V).astype(np.float64)
    if start is not None:
        r, M = r + start, M + np.abs(start)
    return r, M, c


def check_grad(got, r, M, c, dt):
    sums = (c[:, None] + 3) * 2.0 ** -24 * M
    err = np.abs(host64(got) - r)
    assert (err <= sums + STEP[dt] * (np.abs(r) + sums) + TINY[dt]).all(), err.max()


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"),
                                    ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("N,D,V,hot,pad,shift", [
    (1, 1, 1, 0, 0, 0), (1, 136, 7, 0, 0, 0), (2, 515, 3, 0, 0, 0), (33, 8, 1, 0, 0, 0),
    (64, 64, 5, 1.0, 0, 0), (65, 72, 999, 1.0, 8, 0), (129, 1031, 50, 0.5, 3, 1),
    (300, 515, 4099, 0.2, 0, 0), (2500, 264, 700, 0.9, 0, 8), (6001, 40, 33000, 0.4, 0, 0)])
@pytest.mark.parametrize("add", [False, True])
def test_gradient(lib, dt, out, N, D, V, hot, pad, shift, add):
    g = table(N, D, dt, 11, pad, shift)
    y = ids(N, V, 12, hot, invalid=0.1)
    dW = table(V, D, out, 13, pad, shift)
    start = host64(dW) if add else None
    res = lib.embed_backward(g, torch.from_numpy(y).cuda(), V, scale=-0.3, accumulate=add, out=dW)
    assert res is dW
    r, M, c = reference(g, y, V, -0.3, start)
    check_grad(dW, r, M, c, out)
    if not add:
        none = torch.from_numpy(c == 0).cuda()
        if none.any():
            assert_pos_zero("rows of no token", dW[none])
    else:
        assert (host64(dW)[c == 0] == start[c == 0]).all()


def test_gradient_against_differences(lib):
    """The gradient of sum(C * lookup(W)) at W, against central differences of
    the lookup itself: exact for a linear map but for the FP32 roundings."""
    V, D, N = 13, 5, 40
    W, C = table(V, D, "f32", 21), table(N, D, "f32", 22)
    y = torch.from_numpy(ids(N, V, 23, hot=0.3, invalid=0.1)).cuda()
    dW = host64(lib.embed_backward(C, y, V, scale=1.5))
    for v, d in ((0, 0), (V // 2, 3), (V - 1, D - 1), (5, 2)):
        f = []
        for h in (0.5, -0.5):
            P = W.clone()
            P[v, d] += h
            f.append((host64(lib.embed_forward(P, y, scale=1.5)) * host64(C)).sum())
        terms = 1.5 * np.abs(host64(C)).sum() * (np.abs(host64(W)).max() + 0.5)
        assert abs((f[0] - f[1]) - dW[v, d]) <= 8 * 2.0 ** -24 * terms


@pytest.mark.parametrize("N", [0, 1, 50])
def test_gradient_of_no_valid_token(lib, N):
    g = torch.full((N, 24), float("nan"), device="cuda")
    y = torch.full((N,), -100, device="cuda")
    dW = torch.full((9, 32), 5.0, device="cuda")
    lib.embed_backward(g, y, 9, accumulate=True, out=dW[:, :24])
    assert (dW == 5).all()
    lib.embed_backward(g, y, 9, out=dW[:, :24])
    assert_pos_zero("rows of no token", dW[:, :24])
    assert (dW[:, 24:] == 5).all()


@pytest.mark.parametrize("N,hot", [(700, 0.0), (3000, 0.7), (40000, 0.5)])
def test_gradient_bits_and_rows(lib, N, hot):
    """The same bits from run to run, from shards of the vocabulary, and for a
    token whatever the other tokens are."""
    V, D = 3000, 72
    g = table(N, D, "bf16", 31)
    y = ids(N, V, 32, hot, invalid=0.05)
    yc = torch.from_numpy(y).cuda()
    a = lib.embed_backward(g, yc, V)
    assert bits_equal(a, lib.embed_backward(g, yc, V))
    for lo, hi in ((0, 1000), (1000, 1513), (1513, 3000)):
        assert bits_equal(a[lo:hi].contiguous(), lib.embed_backward(g, yc, hi - lo, v0=lo))
    for v in (V // 2, int(y[y >= 0][0])):
        other = np.where(y == v, y, (y * 7 + 1) % V)
        other = np.where((other == v) & (y != v), -100, other)
        b = lib.embed_backward(g, torch.from_numpy(other).cuda(), V)
        assert bits_equal(a[v].contiguous(), b[v].contiguous())


def test_gradient_of_special_values(lib):
    """An infinity or a NaN stays in its own row and column."""
    g = torch.ones(70, 9, device="cuda")
    g[3, 1], g[5, 2], g[69, 8] = float("nan"), float("inf"), -float("inf")
    y = torch.arange(70, device="cuda") % 6
    dW = lib.embed_backward(g, y, 6).cpu()
    assert dW[3, 1].isnan() and dW[5, 2] == float("inf") and dW[69 % 6, 8] == -float("inf")
    dW[3, 1] = dW[5, 2] = dW[69 % 6, 8] = 0
    assert dW.isfinite().all()


def test_offsets_beyond_32_bits(lib):
    """The last row of a table of 2.5e9 elements, read and added into."""
    V, D = 620000, 4096
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    W[-1] = 3.0
    W[V - 1000] = 5.0
    y = torch.tensor([V - 1, V - 1000, V], device="cuda")
    out = lib.embed_forward(W, y)
    assert (out[0] == 3).all() and (out[1] == 5).all() and (out[2] == 0).all()
    g = torch.ones(3, D, dtype=torch.bfloat16, device="cuda")
    lib.embed_backward(g, y, V, accumulate=True, out=W)
    assert (W[-1] == 4).all() and (W[V - 1000] == 6).all()
    del W
    torch.cuda.empty_cache()


def test_streams_and_graphs(lib):
    V, D, N = 2000, 128, 900
    W = table(V, D, "bf16", 41)
    g = table(N, D, "bf16", 42)
    y = torch.from_numpy(ids(N, V, 43, 0.3, 0.1)).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = lib.embed_forward(W, y, stream=s)
    b = lib.embed_backward(g, y, V, stream=s)
    s.synchronize()
    out = torch.empty(N, D, dtype=torch.bfloat16, device="cuda")
    dW = torch.empty(V, D, device="cuda")
    ws = torch.empty(lib.load().ll_embed_workspace_size(N, D, V), dtype=torch.uint8, device="cuda")

    def step():
        lib.embed_forward(W, y, out=out)
        lib.embed_backward(g, y, V, out=dW, workspace=ws)

    step()
    torch.cuda.synchronize()
    assert bits_equal(a, out) and bits_equal(b, dW)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    y.copy_(torch.from_numpy(ids(N, V, 44, 0.6, 0.0)).cuda())
    ws.random_(0, 256)  # a replay may find anything in its workspace
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert bits_equal(out, lib.embed_forward(W, y))
    assert bits_equal(dW, lib.embed_backward(g, y, V))
    assert lib.check_status() == 0


@pytest.mark.parametrize("N", [255, 257, 4095, 4096, 4097, 32767, 32768, 32769, 70001])
@pytest.mark.parametrize("V,invalid", [(1, 0.0), (2, 0.97), (513, 0.0), (511, 0.97), (300000, 0.05),
                                       (140000000, 0.97)])
def test_gradient_where_the_sort_changes(lib, N, V, invalid):
    """Around the sizes at which the sort goes from one block to a cluster and out
    of shared memory, with most tokens dropped, for one to four passes over the digits.
    Small whole numbers, whose sums are exact in any order."""
    D = 8 if V < 1000000 else 1
    rng = np.random.default_rng(N + V)
    y = ids(N, V, N, hot=0.1, invalid=invalid)
    near = rng.random(N) < 0.3  # tokens side by side in the table too
    y = np.where(near & (y >= 0) & (y < V), np.minimum(y % 300, V - 1), y)
    g = torch.from_numpy(rng.integers(-3, 4, (N, D))).to(torch.bfloat16).cuda()
    ok = (y >= 0) & (y < V)
    rows, back = np.unique(y[ok], return_inverse=True)
    want = np.zeros((len(rows), D))
    np.add.at(want, back, host64(g)[ok])
    at = torch.from_numpy(rows).cuda()
    got = lib.embed_backward(g, torch.from_numpy(y).cuda(), V, scale=2.0)
    assert (host64(got[at]) == 2 * want).all()
    got[at] = 0
    assert float(got.abs().max()) == 0
    lib.embed_backward(g, torch.from_numpy(y).cuda(), V, accumulate=True, out=got.fill_(1))
    assert (host64(got[at]) == 1 + want).all()
    got[at] = 1
    assert float(got.min()) == 1 == float(got.max())


@pytest.mark.parametrize("N", [3000, 20000, 60000])
def test_graphs_of_every_sort(lib, N):
    """A captured call of each kind of sort, replayed on other tokens."""
    V, D = 5000, 24
    g = table(N, D, "bf16", 51)
    y = torch.from_numpy(ids(N, V, 52, 0.3, 0.1)).cuda()
    dW, dA = torch.empty(V, D, device="cuda"), torch.zeros(V, D, device="cuda")
    ws = torch.empty(lib.load().ll_embed_workspace_size(N, D, V), dtype=torch.uint8, device="cuda")
    lib.embed_backward(g, y, V, out=dW, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.embed_backward(g, y, V, out=dW, workspace=ws)
        lib.embed_backward(g, y, V, out=dA, workspace=ws, accumulate=True)
    y.copy_(torch.from_numpy(ids(N, V, 53, 0.6, 0.3)).cuda())
    ws.random_(0, 256)
    dA.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = lib.embed_backward(g, y, V)
    assert bits_equal(dW, want) and bits_equal(dA, want)


@pytest.mark.parametrize("dt,out", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("N,D,V,hot", [(1, 4096, 5, 0), (40, 2056, 2, 0), (300, 4096, 9, 0),
                                       (1023, 1031, 40, 0.3), (1024, 2048, 60, 0),
                                       (1024, 515, 1, 0), (1025, 2048, 60, 0)])
def test_few_tokens_added(lib, dt, out, N, D, V, hot):
    """Few tokens added to a table, most of them many times over: right, and the same
    bits from every run."""
    g = table(N, D, dt, 61)
    y = ids(N, V, 62, hot, invalid=0.05)
    yc = torch.from_numpy(y).cuda()
    first = table(V, D, out, 63)
    start = host64(first)
    dW = lib.embed_backward(g, yc, V, scale=0.7, accumulate=True, out=first.clone())
    r, M, c = reference(g, y, V, 0.7, start)
    check_grad(dW, r, M, c, out)
    for _ in range(10):
        assert bits_equal(dW, lib.embed_backward(g, yc, V, scale=0.7, accumulate=True,
                                                 out=first.clone()))


def test_graph_of_few_tokens_added(lib):
    """A captured call for few tokens, replayed on others."""
    N, V, D = 700, 500, 136
    g = table(N, D, "bf16", 71)
    y = torch.from_numpy(ids(N, V, 72, 0.3, 0.1)).cuda()
    dA = torch.zeros(V, D, device="cuda")
    lib.embed_backward(g, y, V, out=dA, accumulate=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.embed_backward(g, y, V, out=dA, accumulate=True)
    y.copy_(torch.from_numpy(ids(N, V, 73, 0.6, 0.3)).cuda())
    dA.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bits_equal(dA, lib.embed_backward(g, y, V, out=torch.zeros_like(dA), accumulate=True))


@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,D,V,hot,pad,shift", [
    (1, 3, 70000, 0, 5, 1), (100, 1, 500000, 0, 0, 0), (777, 72, 20000, 0.1, 8, 0),
    (1023, 1031, 300, 0.3, 3, 1), (1024, 2048, 900, 0, 0, 0), (1024, 136, 1, 0, 0, 0)])
def test_few_tokens_into_a_table_of_their_own(lib, dt, out, N, D, V, hot, pad, shift):
    """Few tokens, every row of the table written, and nothing beside the rows."""
    g = table(N, D, dt, 81)
    y = ids(N, V, 82, hot, invalid=0.05)
    dW = table(V, D, out, 83, pad, shift)
    beside = dW.as_strided((V, dW.stride(0)), (dW.stride(0), 1))[:-1, D:]
    was = beside.clone()
    lib.embed_backward(g, torch.from_numpy(y).cuda(), V, scale=-0.5, out=dW)
    r, M, c = reference(g, y, V, -0.5, None)
    check_grad(dW, r, M, c, out)
    none = torch.from_numpy(c == 0).cuda()
    if none.any():
        assert_pos_zero("rows of no token", dW[none])
    assert bits_equal(beside.contiguous(), was)
