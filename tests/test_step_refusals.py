"""What the embedding, policy-loss and gradient-norm calls refuse: every case
returns before the first CUDA call, so these run on the CPU.  The C ABI gets
made-up pointers that nothing may follow; the binding gets host tensors."""
import ctypes

import pytest
import torch

import cross_entropy_rl_gb300 as ll
from cross_entropy_rl_gb300 import build as B

OK, INVALID, DTYPE, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 4, 5
F32, F16, BF16 = 0, 1, 2
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    B.build()
    return ll.load()


def embed_fwd(L, weight=1 << 20, ldw=64, dtype=BF16, tokens=256, N=4, D=64, V=10, v0=0, scale=1.0,
              out=1 << 30, ldo=64, out_dtype=BF16):
    return L.ll_embed_forward(weight, ldw, dtype, tokens, N, D, V, v0, scale, out, ldo, out_dtype,
                              None)


def embed_bwd(L, g=1 << 20, ldg=64, dtype=BF16, tokens=256, N=4, D=64, V=10, v0=0, scale=1.0,
              acc=0, dW=1 << 30, ldw=64, dw_dtype=F32, ws=1 << 40, ws_bytes=1 << 40):
    return L.ll_embed_backward(g, ldg, dtype, tokens, N, D, V, v0, scale, acc, dW, ldw, dw_dtype,
                               ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=0), OK),
    (dict(N=0, weight=None, tokens=None, out=None), OK),
    (dict(dtype=3), DTYPE), (dict(out_dtype=-1), DTYPE),
    (dict(dtype=F16, out_dtype=BF16), DTYPE), (dict(dtype=BF16, out_dtype=F16), DTYPE),
    (dict(N=-1), SHAPE), (dict(D=0), SHAPE), (dict(V=0), SHAPE), (dict(V=2**31), SHAPE),
    (dict(v0=-1), SHAPE), (dict(v0=2**31 - 260), SHAPE), (dict(ldw=63), SHAPE),
    (dict(ldo=63), SHAPE), (dict(ldw=2**31 + 1), SHAPE),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(weight=None), INVALID), (dict(tokens=None), INVALID), (dict(out=None), INVALID),
    (dict(weight=(1 << 20) + 1), ALIGN), (dict(out=(1 << 30) + 1), ALIGN), (dict(tokens=260), ALIGN),
    (dict(out=(1 << 20) + 2 * 64 * 9 + 126), INVALID),  # the table's last element
    (dict(out=(1 << 20) - 2 * 64 * 4 + 2), INVALID),    # reaches the table's first
])
def test_embed_forward(L, kw, want):
    assert embed_fwd(L, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(N=0, acc=1), OK), (dict(N=0, acc=1, g=None, tokens=None, ws=None, ws_bytes=0), OK),
    (dict(N=0, dW=None), INVALID),
    (dict(dtype=3), DTYPE), (dict(dw_dtype=F16), DTYPE), (dict(dtype=F32, dw_dtype=BF16), DTYPE),
    (dict(N=-1), SHAPE), (dict(D=0), SHAPE), (dict(V=0), SHAPE), (dict(v0=-1), SHAPE),
    (dict(v0=2**31 - 260), SHAPE), (dict(ldg=63), SHAPE), (dict(ldw=63), SHAPE),
    (dict(scale=NAN), INVALID), (dict(scale=-INF), INVALID), (dict(acc=2), INVALID),
    (dict(acc=-1), INVALID), (dict(g=None), INVALID), (dict(tokens=None), INVALID),
    (dict(dW=None), INVALID),
    (dict(g=(1 << 20) + 1), ALIGN), (dict(dW=(1 << 30) + 2), ALIGN), (dict(tokens=4), ALIGN),
    (dict(dW=(1 << 20) + 2 * 64 * 3 + 124), INVALID),
    (dict(ws=None), WORKSPACE), (dict(ws=(1 << 40) + 128), WORKSPACE), (dict(ws_bytes=8), WORKSPACE),
])
def test_embed_backward(L, kw, want):
    assert embed_bwd(L, **kw) == want


def test_embed_workspace(L):
    assert L.ll_embed_workspace_size(0, 64, 10) == 0
    assert L.ll_embed_workspace_size(-1, 64, 10) == 0
    assert L.ll_embed_workspace_size(4, 0, 10) == 0
    need = L.ll_embed_workspace_size(1000, 64, 5000)
    assert need > 0 and need % 256 == 0
    assert embed_bwd(L, N=1000, V=5000, ws_bytes=need - 1) == WORKSPACE


def policy(L, logp=256, old=512, ref=None, adv=768, mask=None, offs=None, B=0, N=4, opt=(),
           reserved=0, stats=1024, grad=1280, ws=1 << 20, ws_bytes=1 << 40):
    o = ll.PolicyOptions(0.2, 0.2, 0.0, 0.0)
    for k, v in dict(opt).items():
        setattr(o, k, v)
    o.reserved[3] = reserved
    return L.ll_policy_loss(logp, old, ref, adv, mask, offs, B, N, ctypes.byref(o), stats, grad, ws,
                            ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(opt=dict(clip_low=1.0)), INVALID), (dict(opt=dict(clip_low=-0.1)), INVALID),
    (dict(opt=dict(clip_low=NAN)), INVALID), (dict(opt=dict(clip_high=-0.1)), INVALID),
    (dict(opt=dict(clip_high=INF)), INVALID), (dict(opt=dict(kl_coef=-1.0)), INVALID),
    (dict(opt=dict(kl_coef=NAN)), INVALID), (dict(opt=dict(kl_coef=0.1)), INVALID),
    (dict(opt=dict(denominator=-1.0)), INVALID), (dict(opt=dict(denominator=INF)), INVALID),
    (dict(opt=dict(denominator=NAN)), INVALID), (dict(reserved=1), INVALID),
    (dict(N=-1), SHAPE), (dict(N=2**31), SHAPE), (dict(B=-1), SHAPE),
    (dict(B=1), INVALID), (dict(offs=256), INVALID), (dict(stats=None), INVALID),
    (dict(logp=None), INVALID), (dict(old=None), INVALID), (dict(adv=None), INVALID),
    (dict(grad=None), INVALID), (dict(logp=258), ALIGN), (dict(ref=258), ALIGN),
    (dict(offs=260, B=2), ALIGN), (dict(stats=1026), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=(1 << 20) + 64), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
])
def test_policy_loss(L, kw, want):
    assert policy(L, **kw) == want


def tensors(*rows):
    arr = (ll.Tensor * max(len(rows), 1))()
    for a, r in zip(arr, rows):
        a.data, a.n, a.dtype, a.reserved = (*r, 0) if len(r) == 3 else r
    return arr, len(rows)


NORM_BAD = [
    ([(1024, 8, 3)], DTYPE), ([(1024, -1, F32)], SHAPE), ([(1024, 2**49, F32)], SHAPE),
    ([(1024, 8, F32, 1)], INVALID), ([(None, 8, F32)], INVALID), ([(1026, 8, F32)], ALIGN),
    ([(1025, 8, BF16)], ALIGN), ([(1024, 8, F32), (2048, 8, 7)], DTYPE),
]


@pytest.mark.parametrize("rows,want", NORM_BAD)
def test_grad_norm(L, rows, want):
    arr, n = tensors(*rows)
    assert L.ll_grad_norm(arr, n, 256, 1 << 20, 1 << 40, None) == want
    assert L.ll_clip_grads(arr, n, 1.0, 0, 256, 1 << 20, 1 << 40, None) == want
    assert L.ll_clip_grads(arr, n, 1.0, 1, 256, None, 0, None) == want


def test_grad_norm_arguments(L):
    arr, n = tensors((1024, 8, F32))
    assert L.ll_grad_norm(None, 1, 256, 1 << 20, 1 << 40, None) == INVALID
    assert L.ll_grad_norm(arr, -1, 256, 1 << 20, 1 << 40, None) == SHAPE
    assert L.ll_grad_norm(arr, n, None, 1 << 20, 1 << 40, None) == INVALID
    assert L.ll_grad_norm(arr, n, 258, 1 << 20, 1 << 40, None) == ALIGN
    assert L.ll_grad_norm(arr, n, 256, None, 1 << 40, None) == WORKSPACE
    assert L.ll_grad_norm(arr, n, 256, (1 << 20) + 8, 1 << 40, None) == WORKSPACE
    need = L.ll_grad_norm_workspace_size(n)
    assert need > 0 and L.ll_grad_norm(arr, n, 256, 1 << 20, need - 1, None) == WORKSPACE
    assert L.ll_grad_norm_workspace_size(-1) == 0
    for bad in (0.0, -1.0, NAN):
        assert L.ll_clip_grads(arr, n, bad, 0, 256, 1 << 20, 1 << 40, None) == INVALID
    assert L.ll_clip_grads(arr, n, 1.0, 2, 256, 1 << 20, 1 << 40, None) == INVALID
    assert L.ll_clip_grads(arr, n, 1.0, 0, 256, None, 0, None) == WORKSPACE


@pytest.mark.parametrize("rows", [
    [(1024, 8, F32), (1024, 8, F32)], [(1024, 8, F32), (1052, 8, F32)],
    [(4096, 1, F32), (1024, 8, BF16), (1038, 1, BF16)],
])
def test_clip_refuses_overlap(L, rows):
    arr, n = tensors(*rows)
    assert L.ll_clip_grads(arr, n, 1.0, 0, 256, 1 << 20, 1 << 40, None) == INVALID
    assert L.ll_clip_grads(arr, n, 1.0, 1, 256, None, 0, None) == INVALID


# ------------------------------------------------------------------ the binding
def test_binding_embed(L):
    W = torch.zeros(10, 16, dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="2-D"):
        ll.embed_forward(W[0], y)
    with pytest.raises(TypeError, match="weight"):
        ll.embed_forward(W.double(), y)
    with pytest.raises(TypeError, match="tokens"):
        ll.embed_forward(W, y.int())
    with pytest.raises(TypeError, match="tokens"):
        ll.embed_forward(W, [1, 2])
    with pytest.raises(ValueError, match="contiguous"):
        ll.embed_forward(W.t(), y)
    with pytest.raises(ValueError, match="contiguous"):
        ll.embed_forward(W[:1].expand(10, 16), y)
    with pytest.raises(ValueError, match="out"):
        ll.embed_forward(W, y, out=torch.zeros(4, 15, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="out_dtype"):
        ll.embed_forward(W, y, out=torch.zeros(4, 16), out_dtype=torch.bfloat16)
    with pytest.raises(ll.LLError):  # host memory
        ll.embed_forward(W, y)
    g = torch.zeros(4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="accumulate"):
        ll.embed_backward(g, y, 10, accumulate=True)
    with pytest.raises(ValueError, match="tokens"):
        ll.embed_backward(g, y[:3], 10)
    with pytest.raises(ValueError, match="out"):
        ll.embed_backward(g, y, 10, out=torch.zeros(9, 16))
    with pytest.raises(ll.LLError):
        ll.embed_backward(g, y, 10, dw_dtype=torch.float16)


def test_binding_policy(L):
    f = torch.zeros(6)
    with pytest.raises(TypeError, match="logp"):
        ll.policy_loss(f.double(), f, f)
    with pytest.raises(ValueError, match="old_logp"):
        ll.policy_loss(f, f[:5], f)
    with pytest.raises(TypeError, match="mask"):
        ll.policy_loss(f, f, f, mask=f)
    with pytest.raises(TypeError, match="seq_offsets"):
        ll.policy_loss(f, f, f, seq_offsets=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="seq_offsets"):
        ll.policy_loss(f, f, f, seq_offsets=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="denominator"):
        ll.policy_loss(f, f, f, denominator=0)
    with pytest.raises(ll.LLError):
        ll.policy_loss(f, f, f)


def test_binding_grads(L):
    a = torch.zeros(6, 4)
    with pytest.raises(TypeError, match="tensor 1"):
        ll.grad_norm([a, [1.0]])
    with pytest.raises(TypeError, match="dtype"):
        ll.grad_norm([a.double()])
    with pytest.raises(ValueError, match="gaps"):
        ll.grad_norm([a[:, :3]])
    with pytest.raises(ValueError, match="gaps"):
        ll.grad_norm([a[:1].expand(6, 4)])
    with pytest.raises(ValueError, match="norm"):
        ll.clip_grads([a], 1.0, norm=torch.zeros(1))
    with pytest.raises(ll.LLError):  # the same memory twice
        ll.clip_grads([a, a.t()], 1.0)
    with pytest.raises(ll.LLError):
        ll.clip_grads([a], 0.0)
