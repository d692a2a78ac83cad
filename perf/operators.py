"""Cases of the operators around the fused linear log-probability in a training step: the embedding
lookup and its gradient, the policy loss that turns logp into grad_logp, and the gradient norm with
clipping.  `run` computes them in plain torch operations, or with `own` through the library."""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # the tokens of one decoding step of 48 requests: launch latency
        dict(name="lookup of one step", op="lookup", N=48, D=4096, V=151936, dtype="bf16",
             out="bf16", scale=64.0, pad=0, invalid=0.0),
        # the prompt and answer tokens of a training step over the largest vocabulary
        dict(name="lookup of a batch", op="lookup", N=32768, D=4096, V=151936, dtype="bf16",
             out="bf16", scale=1.0, pad=0, invalid=0.02),
        # FP32 master weights in a wider buffer, odd width, read as 16-bit activations
        dict(name="lookup, odd rows", op="lookup", N=10007, D=1001, V=32000, dtype="f32",
             out="f16", scale=0.5, pad=6, invalid=0.1),
        # tied weights: added into the FP32 gradient of the output head
        dict(name="gradient, tied", op="lookup_grad", N=32768, D=4096, V=151936, dtype="bf16",
             out="f32", scale=1.0, add=True, hot=0.0, invalid=0.02),
        # untied weights in a 16-bit gradient table, all of it written
        dict(name="gradient, own table", op="lookup_grad", N=4096, D=2048, V=32768, dtype="bf16",
             out="bf16", scale=1.0, add=False, hot=0.0, invalid=0.0),
        # most tokens are one padding token that the user did not mask
        dict(name="gradient, one hot token", op="lookup_grad", N=16384, D=4096, V=32000,
             dtype="f16", out="f32", scale=8.0, add=False, hot=0.6, invalid=0.0),
        # a short ragged batch of odd width
        dict(name="gradient, short", op="lookup_grad", N=301, D=515, V=4099, dtype="f32",
             out="f32", scale=1.0, add=True, hot=0.2, invalid=0.05),
        # one micro-batch, mean over its tokens
        dict(name="policy loss, tokens", op="policy", N=4096, seqs=0, ref=False, mask=0.8),
        # many long answers, mean over the sequences, with the divergence from a reference policy
        dict(name="policy loss, sequences", op="policy", N=1000003, seqs=700, ref=True, mask=0.7),
        # gradients of six wide layers and an FP32 table in flat per-layer buffers: norm alone
        dict(name="norm of large gradients", op="norm", d=2048, layers=6, V=151936, dtype="bf16",
             table="f32"),
        # the same kind of buffers clipped in place
        dict(name="clip of large gradients", op="clip", d=2048, layers=4, V=32768, dtype="bf16",
             table="f32"),
        # a small model: two megabytes in many small tensors
        dict(name="clip of small gradients", op="clip", d=72, layers=6, V=0, dtype="f32",
             table="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "lookup", "lookup_grad", "lookup_grad", "lookup_grad", "policy",
                     "norm", "clip"])
    if op == "lookup":
        dtype = rng.choice(["bf16", "f16", "f32"])
        D = _log(rng, 64, 4096)
        return dict(op=op, N=_log(rng, 1, 32768), D=D if rng.random() < 0.4 else -(-D // 8) * 8,
                    V=_log(rng, 1000, 151936), dtype=dtype,
                    out=rng.choice([dtype, "f32", "bf16" if dtype == "f32" else dtype]),
                    scale=rng.choice([1.0, 0.125, 11.5]), pad=rng.choice([0, 0, 8, 3]),
                    invalid=rng.choice([0.0, 0.05, 0.5]))
    if op == "lookup_grad":
        dtype = rng.choice(["bf16", "f16", "f32"])
        D = _log(rng, 64, 4096)
        return dict(op=op, N=_log(rng, 1, 32768), D=D if rng.random() < 0.4 else -(-D // 8) * 8,
                    V=_log(rng, 1000, 151936), dtype=dtype, out=rng.choice(["f32", "f32", dtype]),
                    scale=rng.choice([1.0, 0.125, 11.5]), add=rng.random() < 0.5,
                    hot=rng.choice([0.0, 0.0, 0.1, 0.7]), invalid=rng.choice([0.0, 0.05]))
    if op == "policy":
        N = _log(rng, 16, 1000000)
        return dict(op=op, N=N, seqs=rng.choice([0, min(N, _log(rng, 1, 2000))]),
                    ref=rng.random() < 0.5, mask=rng.choice([0.3, 0.8, 1.0]))
    return dict(op=op, d=_log(rng, 16, 2048) if rng.random() < 0.7 else 8 * _log(rng, 2, 256),
                layers=rng.randint(1, 4), V=rng.choice([0, _log(rng, 1000, 32768)]),
                dtype=rng.choice(["bf16", "f16", "f32"]), table=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------ inputs
def _tokens(c, g):
    """Token ids: frequencies fall with the rank as in text, ranks spread over the ids; some tokens
    outside the vocabulary, some share one id."""
    N, V = c["N"], c["V"]
    rank = torch.exp(torch.rand(N, device="cuda", generator=g) * math.log(V)).long() - 1
    ids = torch.randperm(V, device="cuda", generator=g)[rank.clamp(0, V - 1)]
    u = torch.rand(N, device="cuda", generator=g)
    ids = torch.where(u < c.get("hot", 0.0), V // 3, ids)
    v = torch.rand(N, device="cuda", generator=g)
    bad = torch.where(v < c["invalid"] / 2, -100, V + 5)
    return torch.where(v < c["invalid"], bad, ids)


def _shapes(c):
    """Gradient shapes of one layer, and whether each is a vector."""
    d = c["d"]
    return [(d, d), (max(d // 4, 1), d), (max(d // 4, 1), d), (d, d), (4 * d, d), (4 * d, d),
            (d, 4 * d), (d,), (d,), (2 * (d // 16) + 1,)]


def _buckets(c, g):
    """One flat buffer per layer, its tensors packed at odd element offsets, and the table's."""
    flat, tensors = [], []
    for layer in range(c["layers"]):
        shapes = _shapes(c)
        total = sum(math.prod(s) + 1 for s in shapes)
        b = torch.randn(total, device="cuda", generator=g).mul_(10.0 ** -(layer % 3)).to(DTYPES[c["dtype"]])
        at = 0
        for s in shapes:
            n = math.prod(s)
            tensors.append(b[at:at + n].view(s))
            b[at + n].zero_()
            at += n + 1
        flat.append(b)
    if c["V"]:
        t = torch.randn(c["V"], c["d"], device="cuda", generator=g).mul_(1e-2).to(DTYPES[c["table"]])
        flat.append(t)
        tensors.append(t)
    return flat, tensors


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "lookup":
        w = torch.randn(c["V"], c["D"] + c["pad"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
        s["weight"] = w[:, :c["D"]]
        s["tokens"] = _tokens(c, g)
    elif c["op"] == "lookup_grad":
        s["tokens"] = _tokens(c, g)
        s["grad"] = torch.randn(c["N"], c["D"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
        if c["add"]:
            s["table"] = torch.randn(c["V"], c["D"], device="cuda", generator=g).to(DTYPES[c["out"]])
    elif c["op"] == "policy":
        N = c["N"]
        s["logp"] = -2.0 * torch.rand(N, device="cuda", generator=g).clamp_min(1e-6).log().neg()
        s["old"] = s["logp"] + 0.15 * torch.randn(N, device="cuda", generator=g)
        s["ref"] = s["logp"] + 0.3 * torch.randn(N, device="cuda", generator=g) if c["ref"] else None
        s["adv"] = torch.randn(N, device="cuda", generator=g)
        s["mask"] = torch.rand(N, device="cuda", generator=g) < c["mask"]
        s["mask"][0] = True
        # masked places hold what an undefined score leaves there
        s["logp"] = torch.where(s["mask"], s["logp"], float("-inf"))
        s["adv"] = torch.where(s["mask"], s["adv"], float("nan"))
        s["offsets"] = None
        if c["seqs"]:
            cut = torch.randint(0, N + 1, (c["seqs"] - 1,), device="cuda", generator=g)
            cut = torch.cat([cut, torch.tensor([0, N], device="cuda")])
            s["offsets"] = cut.sort().values
        s["beta"] = 0.04 if c["ref"] else 0.0
    else:
        s["flat"], s["tensors"] = _buckets(c, g)
        s["bound"] = 1.0
    return s


# ------------------------------------------------------------------ the operators
def _lookup(s):
    c = s["case"]
    out = DTYPES[c["out"]]
    if own:
        import cross_entropy_rl_gb300 as ll
        return ll.embed_forward(s["weight"], s["tokens"], scale=c["scale"], out_dtype=out)
    y = s["tokens"]
    valid = (y >= 0) & (y < c["V"])
    rows = s["weight"][torch.where(valid, y, 0)].float() * c["scale"]
    return torch.where(valid[:, None], rows, 0.0).to(out)


def _lookup_grad(s):
    c = s["case"]
    out = DTYPES[c["out"]]
    if own:
        import cross_entropy_rl_gb300 as ll
        if c["add"]:
            return ll.embed_backward(s["grad"], s["tokens"], c["V"], scale=c["scale"],
                                     accumulate=True, out=s["table"])
        return ll.embed_backward(s["grad"], s["tokens"], c["V"], scale=c["scale"], dw_dtype=out)
    y = s["tokens"]
    valid = (y >= 0) & (y < c["V"])
    rows = torch.where(valid[:, None], s["grad"].float() * c["scale"], 0.0)
    at = torch.where(valid, y, 0)
    if c["add"] and out == torch.float32:
        return s["table"].index_add_(0, at, rows)
    table = s["table"].float() if c["add"] else torch.zeros(c["V"], c["D"], device="cuda")
    table.index_add_(0, at, rows)
    return s["table"].copy_(table) if c["add"] else table.to(out)


CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def _policy(s):
    if own:
        import cross_entropy_rl_gb300 as ll
        return ll.policy_loss(s["logp"], s["old"], s["adv"], ref_logp=s["ref"], mask=s["mask"],
                              seq_offsets=s["offsets"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                              kl_coef=s["beta"])
    # in 64 bits: what lies next to the clipping border, the divergence, which cancels, and the sums
    m = s["mask"]
    logp = torch.where(m, s["logp"], 0.0).double()
    delta = logp - torch.where(m, s["old"], 0.0).double()
    adv = torch.where(m, s["adv"], 0.0)
    clipped = ((adv > 0) & (delta > math.log1p(CLIP_HIGH))) | ((adv < 0) & (delta < math.log1p(-CLIP_LOW)))
    ratio = delta.float().exp()
    loss = -adv * torch.where(clipped, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH), ratio)
    grad = torch.where(clipped, 0.0, -adv * ratio)
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        d = torch.where(m, s["ref"], 0.0).double() - logp
        kl = (torch.expm1(d) - d).float()
        grad = grad - s["beta"] * torch.expm1(d.float())
    if s["offsets"] is None:
        weight = m / m.sum()
    else:
        off = s["offsets"]
        count = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), m.cumsum(0)])[off].diff()
        seq = torch.searchsorted(off, torch.arange(m.numel(), device="cuda"), right=True) - 1
        weight = m / (count[seq].clamp_min(1) * (count > 0).sum())
    policy, div, share = (torch.sum(weight * x, dtype=torch.float64) for x in (loss, kl, clipped))
    stats = torch.stack([policy + s["beta"] * div, policy, div, share])
    return stats.float(), weight * grad


def _norm(s):
    if own:
        import cross_entropy_rl_gb300 as ll
        return ll.grad_norm(s["tensors"])
    return torch.stack([b.float().square().sum().double() for b in s["flat"]]).sum().sqrt().float()


def _clip(s):
    # the gradients are clipped in place: the bound shrinks a little so that every pass clips
    bound = s["bound"]
    s["bound"] = bound * 0.9999
    if own:
        import cross_entropy_rl_gb300 as ll
        return ll.clip_grads(s["tensors"], bound), s["flat"]
    norm = _norm(s)
    coef = torch.clamp(bound / (norm + 1e-6), max=1.0)
    return norm, [b.copy_(b.float() * coef) for b in s["flat"]]


def run(state):
    return {"lookup": _lookup, "lookup_grad": _lookup_grad, "policy": _policy, "norm": _norm,
            "clip": _clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the least work
def _distinct(c):
    """Expected number of distinct tokens: ranks are drawn with frequency ln((r + 2) / (r + 1)) / ln V."""
    r = np.arange(c["V"], dtype=np.float64)
    p = np.log1p(1.0 / (r + 1)) / math.log(c["V"])
    n = c["N"] * (1 - c["invalid"]) * (1 - c.get("hot", 0.0))
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 0.999999))).sum())


def work(case):
    c = case
    if c["op"] == "lookup":
        n = c["N"] * c["D"]
        return {"bytes": 8 * c["N"] + _distinct(c) * c["D"] * SIZE[c["dtype"]] + n * SIZE[c["out"]], "flops": n}
    if c["op"] == "lookup_grad":
        n = c["N"] * (1 - c["invalid"]) * c["D"]
        table = 2 * _distinct(c) if c["add"] else c["V"]
        return {"bytes": 8 * c["N"] + n * SIZE[c["dtype"]] + table * c["D"] * SIZE[c["out"]], "flops": n}
    if c["op"] == "policy":
        return {"bytes": c["N"] * (17 + 4 * c["ref"]) + 8 * c["seqs"], "flops": 20 * c["N"]}
    each = sum(math.prod(x) for x in _shapes(c)) * c["layers"]
    size = each * SIZE[c["dtype"]] + c["V"] * c["d"] * SIZE[c["table"]]
    count = each + c["V"] * c["d"]
    return {"bytes": size, "flops": 2 * count} if c["op"] == "norm" else {"bytes": 2 * size, "flops": 3 * count}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "lookup":
        y = s["tokens"].tolist()
        out = torch.zeros(c["N"], c["D"], dtype=torch.float64, device="cuda")
        good = [n for n, v in enumerate(y) if 0 <= v < c["V"]]
        if good:
            at = torch.tensor(good, device="cuda")
            out[at] = s["weight"].index_select(0, torch.tensor([y[n] for n in good], device="cuda")).double() * c["scale"]
        return out
    if c["op"] == "lookup_grad":
        order = np.argsort(s["tokens"].cpu().numpy(), kind="stable")
        y = s["tokens"].cpu().numpy()[order]
        keep = (y >= 0) & (y < c["V"])
        order, y = order[keep], y[keep]
        table = s["table"].double() if c["add"] else torch.zeros(c["V"], c["D"], dtype=torch.float64, device="cuda")
        if y.size:
            ids, first = np.unique(y, return_index=True)
            last = np.append(first[1:], y.size)
            ids, first, last = (torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (ids, first, last))
            where = torch.from_numpy(order).cuda()
            for j in range(0, c["D"], 512):  # a row's occurrences lie side by side: differences of running sums
                sums = s["grad"][:, j:j + 512].double()[where].cumsum(0)
                sums = torch.cat([torch.zeros_like(sums[:1]), sums])
                table[ids, j:j + 512] += c["scale"] * (sums[last] - sums[first])
        return table
    if c["op"] == "policy":
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        m = s["mask"].cpu().numpy()
        with np.errstate(all="ignore"):
            lp, old, adv = f(s["logp"]), f(s["old"]), f(s["adv"])
            r = np.exp(lp - old)
            low, high = np.minimum(r, 1 + CLIP_HIGH), np.maximum(r, 1 - CLIP_LOW)
            kept = np.where(adv > 0, low, high)  # the smaller of r * adv and the clipped r * adv
            hit = kept != r
            kl, dkl = 0 * r, 0 * r
            if s["ref"] is not None:
                d = f(s["ref"]) - lp
                kl, dkl = np.expm1(d) - d, -np.expm1(d)
            grad = np.where(hit, 0.0, -adv * r) + s["beta"] * dkl
        off = [0, c["N"]] if s["offsets"] is None else s["offsets"].tolist()
        w, full = np.zeros(c["N"]), 0
        for a, b in zip(off[:-1], off[1:]):
            n = int(m[a:b].sum())
            full += n > 0
            w[a:b] = m[a:b] / max(n, 1)
        w /= full
        total = lambda x: float((w[m] * x[m]).sum())  # noqa: E731
        p, k = total(-adv * kept), total(kl)
        out = np.where(m, w * np.where(m, grad, 0.0), 0.0)
        return np.array([p + s["beta"] * k, p, k, total(hit)]), out
    norm = math.sqrt(sum(float(t.double().pow(2).sum()) for t in s["tensors"]))
    if c["op"] == "norm":
        return np.array(norm)
    coef = min(1.0, s["bound"] / (norm + 1e-6))
    return np.array(norm), [b.double().mul_(coef) for b in s["flat"]]
