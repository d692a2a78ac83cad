"""The norm of a list of gradients and clipping by it, against 64 bits.

Bounds (e = 2^-24): the squares are FP32 sums of at most 256 terms, added in 64
bits: 256 e of the sum, so 128 e of its root, and e for the result's rounding.
An element after clipping: 129 e from the norm, 2 e from its sum with 1e-6 and
the division, e from the product, and the half step of its type."""
import math

import numpy as np
import pytest
import torch

from gpu_util import TORCH, bits_equal, host64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
STEP = {torch.float32: E, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}


def norm64(ts):
    return math.sqrt(math.fsum(float((host64(t) ** 2).sum()) for t in ts))


def make(shapes, dts, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, s in enumerate(shapes):
        out.append((torch.randn(s, generator=g) * scale).to(TORCH[dts[i % len(dts)]]).cuda())
    return out


def check(lib, ts, max_norm):
    before = [host64(t) for t in ts]
    ref = math.sqrt(math.fsum(float((b ** 2).sum()) for b in before))
    n = lib.grad_norm(ts)
    assert n.shape == () and abs(float(n) - ref) <= (128 * E + E) * ref
    m = lib.clip_grads(ts, max_norm)
    assert bits_equal(m.view(1), n.view(1))
    coef = min(1.0, max_norm / (ref + 1e-6))
    for t, b in zip(ts, before):
        r = b * coef
        u = STEP[t.dtype]
        assert (np.abs(host64(t) - r) <= (132 * E + u * (1 + 132 * E)) * np.abs(r) + TINY[t.dtype]).all()


MIXED = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("shapes", [
    [(1,)], [(3,), (0,), (1, 1)], [(0,), (0, 5)], [(16384,)], [(16385,), (16383,), (7,)],
    [(33, 515), (1031,), (4, 4, 4), (), (70000,)], [(200001,), (1,), (333, 77)],
    [(n,) for n in range(1, 60)], [(1500, 1003)]])
@pytest.mark.parametrize("dts", [["f32"], ["bf16"], ["f16"], MIXED])
def test_lists(lib, shapes, dts):
    check(lib, make(shapes, dts, 1), 0.7)


def test_no_tensors(lib):
    assert float(lib.grad_norm([])) == 0 and float(lib.clip_grads([], 1.0)) == 0
    assert float(lib.grad_norm([torch.empty(0, device="cuda")])) == 0


@pytest.mark.parametrize("count", [511, 512, 513, 1100])
def test_many_tensors(lib, count):
    """More tensors than one launch takes."""
    check(lib, make([(1 + 37 * (i % 29),) for i in range(count)], MIXED, count), 2.0)


@pytest.mark.parametrize("dt", MIXED)
def test_any_alignment(lib, dt):
    """Views that start and end anywhere in a buffer: nothing next to them changes."""
    buf = make([(5000,)], [dt], 3)[0]
    keep = buf.clone()
    ts, gaps, at = [], [], 0
    for i in range(1, 70):
        ts.append(buf[at + 1:at + 1 + i])
        gaps.append(at)
        at += i + 1
    check(lib, ts, 0.5)
    at_gaps = torch.tensor(gaps, device="cuda")
    assert bits_equal(buf[at_gaps], keep[at_gaps]) and bits_equal(buf[at:], keep[at:])


def test_orders(lib):
    a = make([(40, 30)], ["f32"], 4)[0].t()
    b = make([(2, 8, 5, 6)], ["bf16"], 5)[0].to(memory_format=torch.channels_last)
    check(lib, [a, b], 0.3)


def test_no_clipping_below_the_bound(lib):
    ts = make([(1000,), (33,)], MIXED, 6)
    keep = [t.clone() for t in ts]
    for bound in (1e4, float("inf")):
        lib.clip_grads(ts, bound)
        assert all(bits_equal(a, b) for a, b in zip(ts, keep))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-20, 1e-16, 1e12, 1e18, 1e25, 1e33])
def test_extreme_magnitudes(lib, scale):
    """Squares that leave the FP32 range, alone and beside ordinary ones."""
    ts = make([(50021,), (77,)], ["f32"], 7, scale)
    ref = norm64(ts)
    assert abs(float(lib.grad_norm(ts)) - ref) <= 129 * E * ref + 2.0 ** -149
    both = ts + make([(30000,)], ["f32"], 8)
    ref = norm64(both)
    assert abs(float(lib.grad_norm(both)) - ref) <= 129 * E * ref
    mixed = ts[0].clone()
    mixed[::97] = 1.0
    ref = norm64([mixed])
    assert abs(float(lib.grad_norm([mixed])) - ref) <= 129 * E * ref


def test_zeros_and_special_values(lib):
    z = torch.zeros(40000, dtype=torch.bfloat16, device="cuda")
    assert float(lib.clip_grads([z], 1.0)) == 0 and (z == 0).all()
    t = make([(30001,), (5,)], ["f32"], 9)
    t[0][17] = float("inf")
    assert float(lib.clip_grads(t, 1.0)) == float("inf")
    assert t[0][17].isnan() and (t[0][:17] == 0).all() and (t[1] == 0).all()
    t = make([(30001,), (5,)], ["bf16"], 9)
    t[0][-1] = float("nan")
    assert math.isnan(float(lib.clip_grads(t, 1.0))) and t[1].isnan().all()
    big = torch.full((64,), 3e38, device="cuda")  # a norm beyond FP32
    assert float(lib.grad_norm([big])) == float("inf")


def test_given_norm(lib):
    """Gradients sharded over ranks: the norm of all shards clips each."""
    ts = make([(3000,), (41,), (1030,)], MIXED, 10)
    whole = [t.clone() for t in ts]
    a, b = lib.grad_norm(ts[:1]), lib.grad_norm(ts[1:])
    total = (a.double() ** 2 + b.double() ** 2).sqrt().float()
    for part in (ts[:1], ts[1:]):
        got = lib.clip_grads(part, 0.9, norm=total)
        assert got is total
    n = lib.clip_grads(whole, 0.9)
    if bits_equal(n.view(1), total.view(1)):
        assert all(bits_equal(x, y) for x, y in zip(ts, whole))
    coef = 0.9 / (float(total) + 1e-6)
    assert coef < 1
    for t, w in zip(ts, whole):
        assert np.abs(host64(t) - host64(w)).max() <= 2 * STEP[t.dtype] * np.abs(host64(w)).max()


def test_beyond_32_bits(lib):
    """More than 2^32 elements in one tensor."""
    n = (1 << 32) + 77
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[5], t[1 << 31], t[-1] = 3.0, 4.0, 12.0
    assert float(lib.clip_grads([t], 6.5)) == 13.0
    assert [float(t[i]) for i in (5, 1 << 31, n - 1)] == [1.5, 2.0, 6.0]
    del t
    torch.cuda.empty_cache()


def test_runs_streams_and_graphs(lib):
    ts = make([(70001,), (513, 64), (9,)], MIXED, 11)
    a = lib.grad_norm(ts)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = lib.grad_norm(ts, stream=s)
    s.synchronize()
    assert bits_equal(a.view(1), b.view(1))
    src = [t.clone() for t in ts]
    norm = torch.empty((), device="cuda")
    ws = torch.empty(lib.load().ll_grad_norm_workspace_size(3), dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in ts]
    lib.clip_grads(want, 0.4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.grad_norm(ts, out=norm, workspace=ws)
        lib.clip_grads(ts, 0.4, workspace=ws)
    ws.random_(0, 256)
    for _ in range(2):
        for t, k in zip(ts, src):
            t.copy_(k)
        graph.replay()
    torch.cuda.synchronize()
    assert bits_equal(norm.view(1), a.view(1))
    assert all(bits_equal(x, y) for x, y in zip(ts, want))
