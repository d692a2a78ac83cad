"""The clipped policy loss and its gradient against the definition in 64 bits.

Bounds in FP32 half steps (e = 2^-24), per token with delta = logp - old,
d = ref - logp (both rounded once, so off by at most e of themselves):
  ratio        exp (2 steps = 4 e) of a delta off by e |delta|, one product, one
               rounding of the weight and one of the product with it, one for
               the sum: (8 + |delta|) e |A r|
  divergence   exp(d) - 1: 2 e, d off by e |d| (times exp d), beta's rounding
               and three of the products and the sum: e beta (6 |exp(d) - 1| +
               |d| exp(d)); exp(d) - d - 1 is within 2^-18 of itself (from |d| =
               0.5 on by subtraction, of which 0.106 is left at the least), and
               off by |exp(d) - 1| |d| e for the rounding of d
and for the sums the terms' bounds, and e of the result for its own rounding.
"""
import numpy as np
import pytest
import torch

from gpu_util import assert_pos_zero, bits_equal, host64

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def definition(logp, old, adv, ref=None, mask=None, offs=None, lo=0.2, hi=0.2, beta=0.0, denom=None):
    """(stats, grad, bound of stats, bound of grad), token by token in 64 bits."""
    N = len(logp)
    seq = np.zeros(N, np.int64)
    m = np.ones(N, bool) if mask is None else mask.astype(bool).copy()
    if offs is not None:
        seq[:] = -1
        for b in range(len(offs) - 1):
            seq[offs[b]:offs[b + 1]] = b
        m &= seq >= 0
        count = np.bincount(seq[m], minlength=len(offs) - 1)
        n = float((count > 0).sum()) if denom is None else denom
    else:
        n = float(m.sum()) if denom is None else denom
    grad, gb = np.zeros(N), np.zeros(N)
    stats, sb = np.zeros(4), np.zeros(4)
    for t in np.nonzero(m)[0]:
        x, o, A = float(logp[t]), float(old[t]), float(adv[t])
        w = 1.0 / (n if offs is None else n * count[seq[t]])
        D = x - o
        r = np.exp(D)
        cl = (A > 0 and D > np.log1p(hi)) or (A < 0 and D < np.log1p(-lo))
        bound = (1 + hi) if A > 0 else (1 - lo)
        p = -A * (bound if cl else r)
        grad[t] = 0.0 if cl else -A * r
        pb = (8 + abs(D)) * E * abs(p)
        gb[t] = 0.0 if cl else pb
        k = kb = 0.0
        if ref is not None:
            d = float(ref[t]) - x
            k = np.expm1(d) - d
            kb = 2.0 ** -18 * k + abs(np.expm1(d)) * abs(d) * E
            grad[t] -= beta * np.expm1(d)
            gb[t] += E * beta * (6 * abs(np.expm1(d)) + abs(d) * np.exp(d))
        grad[t] *= w
        gb[t] = gb[t] * w + 2.0 ** -149
        stats += w * np.array([p + beta * k, p, k, float(cl)])
        sb += w * np.array([pb + beta * kb, pb, kb, 0.0])
    return stats, grad, sb + E * np.abs(stats) + 2.0 ** -149, gb


def tokens(N, seed, spread=0.25):
    g = torch.Generator().manual_seed(seed)
    logp = -torch.rand(N, generator=g) * 6
    old = logp + spread * torch.randn(N, generator=g)
    ref = logp + 2 * spread * torch.randn(N, generator=g)
    adv = torch.randn(N, generator=g)
    return [x.cuda() for x in (logp, old, adv, ref)]


def run(lib, logp, old, adv, ref=None, mask=None, offs=None, **kw):
    names = dict(lo="clip_low", hi="clip_high", beta="kl_coef", denom="denominator")
    to = lambda x: None if x is None else torch.as_tensor(x).cuda()  # noqa: E731
    return lib.policy_loss(logp, old, adv, ref_logp=ref, mask=to(mask), seq_offsets=to(offs),
                           **{names[k]: v for k, v in kw.items()})


def check(lib, logp, old, adv, ref=None, **kw):
    stats, grad = run(lib, logp, old, adv, ref, **kw)
    h = [host64(x) if x is not None else None for x in (logp, old, adv, ref)]
    s, g, sb, gb = definition(*h, **kw)
    assert (np.abs(host64(stats) - s) <= sb).all(), (host64(stats), s, sb)
    assert (np.abs(host64(grad) - g) <= gb).all()
    return stats, grad


@pytest.mark.parametrize("N", [1, 2, 31, 33, 256, 1000, 4097, 20011])
@pytest.mark.parametrize("kl", [False, True])
def test_token_mean(lib, N, kl):
    logp, old, adv, ref = tokens(N, N)
    kw = dict(beta=0.07) if kl else {}
    check(lib, logp, old, adv, ref if kl else None, **kw)
    mask = np.random.default_rng(N).random(N) < 0.6
    check(lib, logp, old, adv, ref if kl else None, mask=mask, lo=0.1, hi=0.3, **kw)
    check(lib, logp, old, adv, ref if kl else None, mask=mask, denom=123.5, **kw)


def lengths(kind, N):
    rng = np.random.default_rng(N)
    if kind == "one":
        return [0, N]
    if kind == "singles":
        return list(range(N + 1))
    if kind == "empty":  # empty sequences first, last and in the middle
        return [0, 0, 0, N // 3, N // 3, N // 3, N, N]
    if kind == "partial":  # tokens before the first and after the last
        return [N // 5, N // 2, N // 2, N - N // 7]
    return [0] + sorted(rng.integers(0, N + 1, 40).tolist()) + [N]


@pytest.mark.parametrize("kind", ["one", "singles", "empty", "partial", "ragged"])
@pytest.mark.parametrize("N", [1, 300, 5003])
def test_sequence_mean(lib, kind, N):
    logp, old, adv, ref = tokens(N, N + 1)
    offs = np.array(lengths(kind, N), np.int64)
    mask = np.random.default_rng(N).random(N) < 0.7
    mask[:N // 4] = False  # sequences that the mask leaves empty
    for kw in (dict(), dict(mask=mask), dict(mask=mask, denom=7.0)):
        check(lib, logp, old, adv, ref, offs=offs, beta=0.1, **kw)


def test_many_tokens_and_sequences(lib):
    """Past one pass of every grid: sums against 64 bits, gradients token by token."""
    N, B = 400003, 9000
    logp, old, adv, ref = tokens(N, 5)
    rng = np.random.default_rng(5)
    mask = rng.random(N) < 0.8
    offs = np.array([0] + sorted(rng.integers(0, N + 1, B - 1).tolist()) + [N], np.int64)
    check(lib, logp, old, adv, ref, offs=offs, mask=mask, beta=0.02)
    check(lib, logp, old, adv, ref, mask=mask, beta=0.02)


def test_masked_places_are_not_read(lib):
    N = 1500
    logp, old, adv, ref = tokens(N, 7)
    mask = np.random.default_rng(7).random(N) < 0.5
    stats, grad = check(lib, logp, old, adv, ref, mask=mask, beta=0.1)
    off = torch.from_numpy(~mask).cuda()
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min):
        x = [t.masked_fill(off, bad) for t in (logp, old, adv, ref)]
        s2, g2 = run(lib, *x, mask=mask, beta=0.1)
        assert bits_equal(s2, stats) and bits_equal(g2, grad)
    assert_pos_zero("masked gradients", grad[off])


@pytest.mark.parametrize("offs", [None, [0, 40, 100], [30, 30, 30]])
def test_nothing_left(lib, offs):
    logp, old, adv, ref = tokens(100, 8)
    mask = np.zeros(100, np.uint8)
    offs = None if offs is None else np.array(offs, np.int64)
    stats, grad = run(lib, logp, old, adv, ref, mask=mask, offs=offs, beta=0.1)
    assert_pos_zero("stats", stats)
    assert_pos_zero("grad", grad)
    e = torch.empty(0, device="cuda")
    stats, grad = lib.policy_loss(e, e, e)
    assert_pos_zero("stats", stats)
    assert grad.shape == (0,)


def test_mask_bytes(lib):
    """Any byte that is not 0 counts."""
    logp, old, adv, _ = tokens(64, 9)
    mask = np.arange(64, dtype=np.uint8) * 4
    a = run(lib, logp, old, adv, mask=mask)
    b = run(lib, logp, old, adv, mask=mask != 0)
    assert bits_equal(a[0], b[0]) and bits_equal(a[1], b[1])


def test_border(lib):
    """Values next to the clipping border, where one FP32 step decides: whatever
    the FP32 difference rounds to, the exact one is compared with the border."""
    hi, lo = np.log1p(0.25), np.log1p(-0.25)
    base = np.float32(-7.3)
    old = np.full(400, base, np.float32)
    logp = np.empty(400, np.float32)
    for i in range(200):
        x = np.float32(base + np.float32(hi))
        y = np.float32(base + np.float32(lo))
        for _ in range(abs(i - 100)):
            x = np.nextafter(x, np.float32(np.sign(i - 100) * 1e9))
            y = np.nextafter(y, np.float32(np.sign(i - 100) * 1e9))
        logp[i], logp[200 + i] = x, y
    adv = np.r_[np.ones(200), -np.ones(200)].astype(np.float32)
    t = [torch.from_numpy(x).cuda() for x in (logp, old, adv)]
    _, grad = check(lib, *t, lo=0.25, hi=0.25)
    D = logp.astype(np.float64) - old
    want = np.r_[D[:200] > hi, D[200:] < lo]
    assert ((host64(grad) == 0) == want).all() and 0 < want.sum() < 400


def test_no_advantage_and_extremes(lib):
    """A zero advantage has no policy part even where the ratio overflows; a
    ratio that overflows is clipped for A > 0 and infinite for A < 0."""
    logp = torch.tensor([0.0, 0.0, 0.0, -200.0, -200.0], device="cuda")
    old = torch.tensor([-200.0, -200.0, -200.0, 0.0, 0.0], device="cuda")
    adv = torch.tensor([0.0, 1.0, -1.0, 1.0, -1.0], device="cuda")
    for i, (p, g) in enumerate(((0, 0), (-1.2, 0), (np.inf, np.inf), (0, 0), (0.8, 0))):
        s, grad = run(lib, logp[i:i + 1], old[i:i + 1], adv[i:i + 1])
        assert float(grad[0]) == g and (float(s[1]) == p if not p or np.isinf(p) else
                                        abs(float(s[1]) - p) < 1e-6)


def test_small_divergences(lib):
    """exp(d) - d - 1 where it is far below the rounding of exp(d)."""
    d = torch.tensor([1e-6, -1e-5, 3e-4, -1e-3, 0.02, -0.1, 0.49, -0.5, 0.51, 3.0], device="cuda")
    logp = torch.zeros_like(d)
    for i in range(len(d)):
        s = run(lib, logp[i:i + 1], logp[i:i + 1], logp[i:i + 1], d[i:i + 1])[0]
        x = float(d[i])
        want = x * x / 2 + x ** 3 / 6 + x ** 4 / 24 if abs(x) < 1e-3 else np.expm1(x) - x
        assert abs(float(s[2]) - want) <= 2.0 ** -18 * want


def test_gradient_against_differences(lib):
    """The gradient from central differences of the 64-bit definition."""
    N = 60
    logp, old, adv, ref = tokens(N, 11)
    offs, mask = np.array([0, 10, 10, 41, 60], np.int64), np.random.default_rng(1).random(N) < 0.8
    _, grad = run(lib, logp, old, adv, ref, mask=mask, offs=offs, beta=0.3)
    h = [host64(x) for x in (logp, old, adv, ref)]
    D = h[0] - h[1]
    for t in range(N):
        if min(abs(D[t] - np.log1p(0.2)), abs(D[t] - np.log1p(-0.2))) < 1e-3:
            continue  # a difference across the border is no derivative
        f = []
        for step in (1e-4, -1e-4):
            x = h[0].copy()
            x[t] += step
            f.append(definition(x, *h[1:], mask=mask, offs=offs, beta=0.3)[0][0])
        assert abs((f[0] - f[1]) / 2e-4 - float(grad[t])) <= 1e-6 + 1e-5 * abs(float(grad[t]))


def test_runs_streams_and_graphs(lib):
    N = 5000
    logp, old, adv, ref = tokens(N, 12)
    offs = torch.tensor(lengths("ragged", N), device="cuda")
    kw = dict(ref_logp=ref, seq_offsets=offs, kl_coef=0.1)
    a = lib.policy_loss(logp, old, adv, **kw)
    b = lib.policy_loss(logp, old, adv, **kw)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c = lib.policy_loss(logp, old, adv, stream=s, **kw)
    s.synchronize()
    out = (torch.empty(4, device="cuda"), torch.empty(N, device="cuda"))
    ws = torch.empty(lib.load().ll_policy_workspace_size(N, len(offs) - 1), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.policy_loss(logp, old, adv, out=out, workspace=ws, **kw)
    ws.random_(0, 256)  # a replay may find anything in its workspace
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x in (b, c, out):
        assert bits_equal(a[0], x[0]) and bits_equal(a[1], x[1])
    adv.neg_()
    graph.replay()
    d = lib.policy_loss(logp, old, adv, **kw)
    assert bits_equal(d[0], out[0]) and bits_equal(d[1], out[1]) and not bits_equal(a[1], out[1])


@pytest.mark.parametrize("kind", ["one", "few", "thousands", "short", "clumps", "partial"])
@pytest.mark.parametrize("N", [5003, 1000003])
def test_every_token_has_its_sequence(lib, kind, N):
    """Weights alone: with a ratio of 1 and an advantage of -1 a token's gradient is
    1 / (tokens of its sequence x sequences), an FP32 quotient of a rounded one."""
    rng = np.random.default_rng(N)
    cuts = {"one": 0, "few": N // 1500, "thousands": N // 60, "short": N // 2, "clumps": N // 400,
            "partial": 50}[kind]
    at = np.sort(rng.integers(0, N + 1, cuts))
    if kind == "clumps":  # a hundred empty sequences at every cut
        at = np.repeat(at, 101)
    offs = np.concatenate([[0], at, [N]]) if kind != "partial" else at
    mask = rng.random(N) < 0.7
    seq = np.searchsorted(offs, np.arange(N), side="right") - 1
    ok = mask & (seq >= 0) & (seq < len(offs) - 1)
    count = np.bincount(seq[ok], minlength=len(offs) - 1)
    want = np.where(ok, 1.0 / (np.maximum(count[np.clip(seq, 0, len(offs) - 2)], 1) *
                               float((count > 0).sum())), 0.0)
    x = torch.zeros(N, device="cuda")
    stats, grad = run(lib, x, x, x - 1, mask=mask, offs=offs.astype(np.int64))
    assert (np.abs(host64(grad) - want) <= 2.0 ** -23 * 1.001 * want).all()
    assert abs(float(stats[0]) - 1) <= 2.0 ** -23 and float(stats[3]) == 0
