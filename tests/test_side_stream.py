"""Memory of a call on a stream of the caller's.  The allocator hands out a block that
was freed on the current stream while work queued there still uses it, so such a call
takes what it allocates from its own stream.  On the CPU with a fake allocator."""
import contextlib

import pytest
import torch

import cross_entropy_rl_gb300 as ll

DEVICE = torch.device("cuda", 0)


class Allocation:
    is_cuda = True

    def __init__(self, pool):
        self.pool, self.users = pool, []

    def record_stream(self, stream):
        self.users.append(stream)


@pytest.fixture
def allocations(monkeypatch):
    current, made = ["current"], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(*shape, dtype=None, device=None):
        assert device == DEVICE
        made.append(Allocation(current[-1]))
        return made[-1]

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    return made


def test_outputs_come_from_the_stream_that_writes_them(allocations):
    t = ll._new((3, 4), torch.float32, DEVICE, "side")
    assert t.pool == "side"
    assert t.users == ["current"]  # the caller may drop them while that stream reads


def test_gradients_and_workspaces_of_the_linear_calls(allocations, monkeypatch):
    monkeypatch.setattr(ll, "_need", lambda *a, **k: None)
    bf16, f32 = torch.bfloat16, torch.float32
    grads = ll._grad_outputs(None, True, True, True, 4, 8, 16, bf16, None, None, DEVICE, "side")
    assert [t.pool for t in grads[:3]] == ["side"] * 3 and grads[3:] == (bf16, f32)
    assert ll._workspace(1000, DEVICE, "side").pool == "side"


def test_workspaces_come_from_the_stream_that_uses_them(allocations):
    t = ll._scratch(None, 1000, DEVICE, "side")
    assert t.pool == "side"
    assert t.users == []  # nothing else ever touches it


@pytest.mark.parametrize("stream", [None, "current"])
def test_the_current_stream_needs_nothing(allocations, stream):
    for t in (ll._new((3, 4), torch.float32, DEVICE, stream), ll._scratch(None, 1000, DEVICE, stream)):
        assert t.pool == "current" and t.users == []


def test_the_current_stream_without_the_private_getter(monkeypatch):
    """The handle comes from the public call where torch lacks the quicker one."""
    class Stream:
        cuda_stream = 4711

    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: asked.append(device) or Stream)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert ll._stream_of(DEVICE, None) == 4711 and asked == [DEVICE]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    assert ll._stream_of(DEVICE, None) == 100 and asked == [DEVICE]
