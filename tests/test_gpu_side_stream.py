"""Calls on a stream of the caller's while the current stream is busy: what they
allocate is that stream's memory, not a block that the current stream still uses."""
import pytest
import torch

import cross_entropy_rl_gb300 as ll
from gpu_util import bits_equal

pytestmark = pytest.mark.gpu


def pool_of(t):
    """The stream whose memory holds t."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's memory")


def calls():
    """name -> (call(stream) -> tensors that it allocates)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    N, D, V = 3000, 512, 2000
    W = torch.randn(V, D, device="cuda", generator=g)
    y = torch.randint(0, V, (N,), device="cuda", generator=g)
    x = torch.randn(N, D, device="cuda", generator=g)
    logp = -torch.rand(N, device="cuda", generator=g)
    old, adv = logp + 0.1, torch.randn(N, device="cuda", generator=g)
    offs = torch.tensor([0, 700, N], device="cuda")
    grads = [x, W]
    h, Wb = x.bfloat16(), (W * D ** -0.5).bfloat16()
    lse = ll.forward(h, Wb, None, y)[1]
    z = torch.randn(N, V, device="cuda", generator=g)
    zl = ll.logits_fwd(z, y)[1]
    parts = ll.forward_shard(h, Wb, None, y, 0, V)
    return {
        "embed_forward": lambda s: [ll.embed_forward(W, y, stream=s)],
        "embed_backward": lambda s: [ll.embed_backward(x, y, V, stream=s)],
        "policy_loss": lambda s: list(ll.policy_loss(logp, old, adv, seq_offsets=offs, stream=s)),
        "forward": lambda s: list(ll.forward(h, Wb, None, y, stream=s)),
        "backward": lambda s: list(ll.backward(adv, h, Wb, None, y, lse, stream=s))[:2],
        "forward_backward": lambda s: list(ll.forward_backward(adv, h, Wb, None, y, need_db=True,
                                                               stream=s)),
        "logits_fwd": lambda s: list(ll.logits_fwd(z, y, stream=s)),
        "logits_bwd": lambda s: [ll.logits_bwd(adv, z, y, zl, stream=s)],
        "logits_fwd_bwd": lambda s: list(ll.logits_fwd_bwd(adv, z, y, stream=s)),
        "forward_shard": lambda s: list(ll.forward_shard(h, Wb, None, y, 0, V, stream=s)),
        "lse_merge": lambda s: list(ll.lse_merge(*parts, y, V, stream=s)),
        "backward_shard": lambda s: list(ll.backward_shard(adv, h, Wb, None, y, lse, 0, V,
                                                           stream=s))[:2],
        "sum_ordered": lambda s: [ll.sum_ordered(x, stream=s)],
        "grad_norm": lambda s: [ll.grad_norm(grads, stream=s)],
        "clip_grads": lambda s: [ll.clip_grads(grads, float("inf"), stream=s)],
    }


@pytest.mark.parametrize("name", [
    "embed_forward", "embed_backward", "policy_loss", "grad_norm", "clip_grads", "forward", "backward",
    "forward_backward", "logits_fwd", "logits_bwd", "logits_fwd_bwd", "forward_shard", "lse_merge",
    "backward_shard", "sum_ordered"])
def test_memory_of_a_call_on_another_stream(lib, monkeypatch, name):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []  # a call's scratch, held as long as what is queued here
    new = ll._new

    def keep(*a, **k):
        kept.append(new(*a, **k))
        return kept[-1]

    monkeypatch.setattr(ll, "_new", keep)
    call(side)  # the first memory of a stream and the first use of a kernel wait for the device
    torch.cuda.synchronize()
    sizes = [t.untyped_storage().nbytes() for t in kept]
    kept.clear()
    # freed here just before, in every size that the call allocates, and still written
    junk = [torch.full((n,), 0, dtype=torch.uint8, device="cuda") for n in sizes]
    at = [t.data_ptr() for t in junk]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    for t in junk:
        t.fill_(255)
    del junk, t
    got = call(side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()  # its writes are still to come
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert bits_equal(a.reshape(-1), b.reshape(-1))
    assert kept and all(pool_of(t) == side.cuda_stream for t in kept)
    assert not {t.data_ptr() for t in kept} & set(at)


def test_the_current_stream_given(lib):
    """stream= the current stream is the call without it."""
    call = calls()["policy_loss"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got, plain = call(side), call(None)
        assert all(pool_of(t) == side.cuda_stream for t in got + plain)
        assert all(bits_equal(a, b) for a, b in zip(got, plain))


def test_captured_on_a_branch(lib):
    """A call on a stream that joins a capture: its memory belongs to the graph."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(5000, device="cuda", generator=g)
    old, adv = x - 0.1, torch.randn(5000, device="cuda", generator=g)
    want = ll.policy_loss(x, old, adv)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = ll.policy_loss(x, old, adv, stream=side)
        here.wait_stream(side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(bits_equal(a, b) for a, b in zip(got, want))
