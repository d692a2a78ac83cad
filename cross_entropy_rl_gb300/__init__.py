"""GB300-native fused linear log-probability: thin Python binding.

The computation runs in the CUDA library ``_lib/libll_gb300.so`` built from
``csrc/`` (C ABI in ``include/ll_linear_logp.h``).  This module only
marshals arguments: it takes torch tensors, allocates outputs and the scratch
workspace with torch (the library itself never allocates), and passes raw
pointers plus the current CUDA stream.  There is no fallback: every call
raises when the library is missing or a call returns an error status.

    import cross_entropy_rl_gb300 as ll
    logp, lse = ll.forward(hidden, weight, bias, targets)
    dh, dW, db = ll.backward(grad_logp, hidden, weight, bias, targets, lse)
"""
from __future__ import annotations

import array
import ctypes
import os

__all__ = [
    "LLError", "load", "lib", "forward", "backward", "forward_backward", "logits_fwd",
    "logits_bwd", "logits_fwd_bwd", "shard_segments", "forward_shard", "lse_merge",
    "backward_shard", "SEGMENT_COLS",
    "embed_forward", "embed_backward", "policy_loss", "grad_norm", "clip_grads",
    "FP4Matrix", "fp4_quantize", "fp4_dequantize", "fp4_linear", "sample",
    "workspace_size", "check_status", "DTYPE_CODES", "EXPORTS",
]

_LIB = None
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libll_gb300.so")

# ll_dtype codes of the C ABI
LL_F32, LL_F16, LL_BF16 = 0, 1, 2
# vocab entries per LSE segment; vocab shards start on a multiple of it
SEGMENT_COLS = 1024

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_size = ctypes.c_size_t
_c_float = ctypes.c_float

# name -> (restype, argtypes): every symbol the header declares
EXPORTS = {
    "ll_status_string": (ctypes.c_char_p, [_c_int]),
    "ll_version": (_c_int, []),
    "ll_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int]),
    "ll_forward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_int,
                            _c_p, _c_p, _c_p, _c_size, _c_p]),
    "ll_backward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                             _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                             _c_p, _c_int, _c_p, _c_size, _c_p]),
    "ll_forward_backward": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                                     _c_int, _c_p, _c_p, _c_int, _c_int, _c_int, _c_p, _c_int,
                                     _c_p, _c_int, _c_p, _c_int, _c_p, _c_size, _c_p]),
    "logits_logp_fwd": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "logits_logp_bwd": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_p, _c_p, _c_i64, _c_i64,
                                 _c_p, _c_p]),
    "logits_logp_fwd_bwd": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_p,
                                     _c_p, _c_p, _c_p]),
    "ll_shard_segments": (_c_i64, [_c_i64]),
    "ll_workspace_size_shard": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                                          _c_int]),
    "ll_forward_shard": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_i64,
                                  _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p, _c_size, _c_p, _c_p]),
    "ll_lse_merge": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_i64, _c_p,
                              _c_p, _c_p]),
    "ll_backward_shard": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                                   _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_p,
                                   _c_int, _c_p, _c_int, _c_p, _c_int, _c_p, _c_size, _c_p,
                                   _c_p]),
    "ll_forward_ex": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_int,
                               _c_p, _c_p, _c_p, _c_size, _c_p, _c_p]),
    "ll_backward_ex": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                                _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                                _c_p, _c_int, _c_p, _c_size, _c_p, _c_p]),
    "ll_forward_backward_ex": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64,
                                        _c_int, _c_p, _c_p, _c_int, _c_int, _c_int, _c_p,
                                        _c_int, _c_p, _c_int, _c_p, _c_int, _c_p, _c_size,
                                        _c_p, _c_p]),
    "logits_logp_fwd_ex": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_p, _c_p,
                                    _c_p, _c_p]),
    "logits_logp_bwd_ex": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_p, _c_p, _c_i64, _c_i64,
                                    _c_p, _c_p, _c_p]),
    "logits_logp_fwd_bwd_ex": (_c_int, [_c_p, _c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64,
                                        _c_p, _c_p, _c_p, _c_p, _c_p]),
    "ll_check_status": (_c_int, [_c_p]),
    "ll_set_wait_limit_ns": (None, [_c_i64]),
    "ll_debug_unsatisfied_wait": (_c_int, [_c_p, _c_p]),
    "ll_forward_noalloc": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_int,
                                    _c_p, _c_p, _c_p]),
    "ll_launch_count": (ctypes.c_longlong, []),
    "ll_profile_enable": (None, [_c_int]),
    "ll_profile_summary": (_c_int, [ctypes.c_char_p, _c_size]),
    "ll_sum_ordered": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_int, _c_p, _c_p]),
    "ll_embed_forward": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_i64, _c_i64,
                                  _c_float, _c_p, _c_i64, _c_int, _c_p]),
    "ll_embed_workspace_size": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "ll_embed_backward": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_i64, _c_i64,
                                   _c_float, _c_int, _c_p, _c_i64, _c_int, _c_p, _c_size, _c_p]),
    "ll_policy_workspace_size": (_c_size, [_c_i64, _c_i64]),
    "ll_policy_loss": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p,
                                _c_p, _c_p, _c_size, _c_p]),
    "ll_grad_norm_workspace_size": (_c_size, [_c_i64]),
    "ll_grad_norm": (_c_int, [_c_p, _c_i64, _c_p, _c_p, _c_size, _c_p]),
    "ll_clip_grads": (_c_int, [_c_p, _c_i64, _c_float, _c_int, _c_p, _c_p, _c_size, _c_p]),
    "ll_fp4_row_bytes": (_c_size, [_c_i64]),
    "ll_fp4_scale_bytes": (_c_size, [_c_i64, _c_i64, _c_int]),
    "ll_fp4_quantize": (_c_int, [_c_p, _c_i64, _c_int, _c_i64, _c_i64, _c_int, _c_p, _c_int,
                                 _c_p, _c_p, _c_p]),
    "ll_fp4_dequantize": (_c_int, [_c_p, _c_p, _c_p, _c_i64, _c_i64, _c_int, _c_p, _c_i64, _c_int,
                                   _c_p]),
    "ll_fp4_linear": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64,
                               _c_i64, _c_int, _c_p, _c_i64, _c_int, _c_p]),
    "ll_sample_workspace_size": (_c_size, [_c_i64, _c_i64, _c_int]),
    "ll_sample": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p,
                           _c_p, _c_size, _c_p]),
}


class Options(ctypes.Structure):
    """ll_options of the C ABI."""
    _fields_ = [("temperature", ctypes.c_float), ("split_s", ctypes.c_int),
                ("reserved", ctypes.c_int * 6)]


SPLIT_MODES = {"auto": 0, "always": 1, "never": 2}


def _split_code(split_s) -> int:
    """ll_options.split_s of a binding argument: "auto" (or None, the
    default), "always" (or True) or "never" (or False)."""
    if split_s is None:
        return 0
    if isinstance(split_s, bool):
        return 1 if split_s else 2
    if split_s not in SPLIT_MODES:
        raise ValueError(f"split_s must be one of {sorted(SPLIT_MODES)}, True, False or None")
    return SPLIT_MODES[split_s]


def _opts(temperature=1.0, split_s="auto"):
    """ll_options pointer for a call (None when every option is default)."""
    t = 1.0 if temperature is None else float(temperature)
    if not t > 0:
        raise ValueError("temperature must be > 0")
    code = _split_code(split_s)
    if t == 1.0 and code == 0:
        return None
    return ctypes.byref(Options(temperature=t, split_s=code))


class LLError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = "?"
        if _LIB is not None:
            msg = _LIB.ll_status_string(status).decode()
        super().__init__(f"{fn} failed: status {status} ({msg})")
        self.status = status


def load(path: str | None = None):
    """Load the shared library (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library not built: {path} is missing "
            "(run `python -m cross_entropy_rl_gb300.build`)")
    lib_ = ctypes.CDLL(path)
    for name, (res, args) in EXPORTS.items():
        f = getattr(lib_, name)
        f.restype = res
        f.argtypes = args
    _LIB = lib_
    return _LIB


def lib():
    return load()


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _code(dtype) -> int:
    torch = _torch()
    m = {torch.float32: LL_F32, torch.float16: LL_F16, torch.bfloat16: LL_BF16}
    if dtype not in m:
        raise TypeError(f"unsupported dtype {dtype}")
    return m[dtype]


def DTYPE_CODES():
    torch = _torch()
    return {torch.float32: LL_F32, torch.float16: LL_F16, torch.bfloat16: LL_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    if stream is None and not torch.cuda.is_available():
        return ctypes.c_void_p(None)  # the call itself then fails: no device memory
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, st: int):
    if st != 0:
        raise LLError(fn, st)


def workspace_size(N, D, V, dtype, token_chunks=0, backward=False, need_db=False) -> int:
    code = dtype if isinstance(dtype, int) else _code(dtype)
    return int(load().ll_workspace_size(N, D, V, code, token_chunks, int(backward),
                                        int(bool(need_db))))


def _need(t, name, shape, dtype=None, device=None, dtypes=None):
    """Raise unless tensor t is contiguous, on `device`, of `shape` and dtype.

    The C ABI receives bare pointers, so every buffer it reads or writes is
    checked here, where the sizes are still known."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.numel() and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_linear(hidden, weight, bias, targets):
    torch = _torch()
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden and weight must be 2-D")
    N, D = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    _need(hidden, "hidden", (N, D), device=dev,
          dtypes=(torch.float32, torch.float16, torch.bfloat16))
    _need(weight, "weight", (V, D), hidden.dtype, dev)
    if bias is not None:
        _need(bias, "bias", (V,), hidden.dtype, dev)
    _need(targets, "targets", (N,), torch.int64, dev)
    return N, D, V, dev


def _new(shape, dtype, device, stream, scratch=False):
    """A new tensor for a call on the current stream, or on `stream`.

    The allocator hands a block that was freed on a stream to that stream alone:
    work queued there may still use it.  So what `stream` writes comes from its
    own memory.  The caller may use it on the current stream and then drop it, so
    the allocator also waits for that one, unless it is scratch of the call."""
    torch = _TORCH or _torch()
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    if stream == here:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(here)
    return t


def _workspace(nbytes, device, stream):
    return _new((max(int(nbytes), 256),), _torch().uint8, device, stream, scratch=True)


def _grad_outputs(out, need_dh, need_dw, need_db, N, D, V, op_dtype, dh_dtype, dw_dtype, dev,
                  stream):
    """Gradient buffers (given or allocated) and their dtypes.  A given
    buffer's dtype decides; an explicit dtype that disagrees with it raises."""
    torch = _torch()
    if out is not None:
        dh, dW, db = out
        if dh is not None:
            if dh_dtype is not None and dh_dtype != dh.dtype:
                raise TypeError("dh_dtype disagrees with the given grad_hidden")
            dh_dtype = dh.dtype
        if dW is not None or db is not None:
            given = (dW if dW is not None else db).dtype
            if dw_dtype is not None and dw_dtype != given:
                raise TypeError("dw_dtype disagrees with the given grad_weight / grad_bias")
            dw_dtype = given
    dh_dtype = op_dtype if dh_dtype is None else dh_dtype
    dw_dtype = torch.float32 if dw_dtype is None else dw_dtype
    if out is None:
        dh = _new((N, D), dh_dtype, dev, stream) if need_dh else None
        dW = _new((V, D), dw_dtype, dev, stream) if need_dw else None
        db = _new((V,), dw_dtype, dev, stream) if need_db else None
    if need_dh:
        _need(dh, "grad_hidden", (N, D), dh_dtype, dev)
    if need_dw:
        _need(dW, "grad_weight", (V, D), dw_dtype, dev)
    if need_db:
        _need(db, "grad_bias", (V,), dw_dtype, dev)
    return dh, dW, db, dh_dtype, dw_dtype


def forward(hidden, weight, bias, targets, *, temperature=1.0, workspace=None, out=None,
            stream=None):
    """(logp [N] fp32, lse [N] fp32) of z = hidden . weight^T (+ bias); with a
    temperature T the distribution is softmax(z / T)."""
    torch = _torch()
    L = load()
    N, D, V, dev = _check_linear(hidden, weight, bias, targets)
    code = _code(hidden.dtype)
    if out is None:
        logp = _new((N,), torch.float32, dev, stream)
        lse = _new((N,), torch.float32, dev, stream)
    else:
        logp, lse = out
    _need(logp, "logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    ws_need = L.ll_workspace_size(N, D, V, code, 0, 0, 0)
    if workspace is None:
        workspace = _workspace(ws_need, dev, stream)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    st = L.ll_forward_ex(_ptr(hidden), _ptr(weight), _ptr(bias), _ptr(targets), N, D, V, code,
                         _ptr(logp), _ptr(lse), _ptr(workspace), workspace.numel(),
                         _opts(temperature), _stream(stream))
    _check("ll_forward", st)
    return logp, lse


def backward(grad_logp, hidden, weight, bias, targets, lse, *, need_dh=True, need_dw=True,
             need_db=None, dh_dtype=None, dw_dtype=None, token_chunks=0, temperature=1.0,
             split_s="auto", workspace=None, out=None, stream=None):
    """(grad_hidden, grad_weight, grad_bias); entries not requested are None.

    dw_dtype defaults to float32; grad_bias uses dw_dtype.
    """
    torch = _torch()
    L = load()
    N, D, V, dev = _check_linear(hidden, weight, bias, targets)
    code = _code(hidden.dtype)
    if need_db is None:
        need_db = bias is not None
    _need(grad_logp, "grad_logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    dh, dW, db, dh_dtype, dw_dtype = _grad_outputs(out, need_dh, need_dw, need_db, N, D, V,
                                                   hidden.dtype, dh_dtype, dw_dtype, dev,
                                                   stream)
    ws_need = L.ll_workspace_size(N, D, V, code, token_chunks, 1,
                                  int(bool(need_db)) | (_split_code(split_s) << 1))
    if workspace is None:
        workspace = _workspace(ws_need, dev, stream)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    st = L.ll_backward_ex(_ptr(grad_logp), _ptr(hidden), _ptr(weight), _ptr(bias),
                          _ptr(targets), _ptr(lse), N, D, V, code, int(bool(need_dh)),
                          int(bool(need_dw)), int(bool(need_db)), _ptr(dh), _code(dh_dtype),
                          _ptr(dW), _code(dw_dtype), _ptr(db), int(token_chunks),
                          _ptr(workspace), workspace.numel(), _opts(temperature, split_s),
                          _stream(stream))
    _check("ll_backward", st)
    return dh, dW, db


def forward_backward(grad_logp, hidden, weight, bias, targets, *, need_dh=True, need_dw=True,
                     need_db=None, dh_dtype=None, dw_dtype=None, token_chunks=0,
                     temperature=1.0, split_s="auto", workspace=None, out=None, stream=None):
    """(logp, lse, grad_hidden, grad_weight, grad_bias) in one call, for a
    grad_logp known before the forward; bitwise equal to forward + backward."""
    torch = _torch()
    L = load()
    N, D, V, dev = _check_linear(hidden, weight, bias, targets)
    code = _code(hidden.dtype)
    if need_db is None:
        need_db = bias is not None
    _need(grad_logp, "grad_logp", (N,), torch.float32, dev)
    if out is not None:
        logp, lse, dh, dW, db = out
        grads = (dh, dW, db)
    else:
        logp = _new((N,), torch.float32, dev, stream)
        lse = _new((N,), torch.float32, dev, stream)
        grads = None
    _need(logp, "logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    dh, dW, db, dh_dtype, dw_dtype = _grad_outputs(grads, need_dh, need_dw, need_db, N, D, V,
                                                   hidden.dtype, dh_dtype, dw_dtype, dev,
                                                   stream)
    ws_need = L.ll_workspace_size(N, D, V, code, token_chunks, 2,
                                  int(bool(need_db)) | (_split_code(split_s) << 1))
    if workspace is None:
        workspace = _workspace(ws_need, dev, stream)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    st = L.ll_forward_backward_ex(_ptr(grad_logp), _ptr(hidden), _ptr(weight), _ptr(bias),
                                  _ptr(targets), N, D, V, code, _ptr(logp), _ptr(lse),
                                  int(bool(need_dh)), int(bool(need_dw)), int(bool(need_db)),
                                  _ptr(dh), _code(dh_dtype), _ptr(dW), _code(dw_dtype),
                                  _ptr(db), int(token_chunks), _ptr(workspace),
                                  workspace.numel(), _opts(temperature, split_s),
                                  _stream(stream))
    _check("ll_forward_backward", st)
    return logp, lse, dh, dW, db


def logits_fwd(logits, targets, V=None, *, temperature=1.0, out=None, stream=None):
    """(logp, lse) from logits [N, ld]; columns >= V (default ld) ignored."""
    torch = _torch()
    L = load()
    N, ld = logits.shape
    V = ld if V is None else V
    dev = logits.device
    _need(logits, "logits", (N, ld), device=dev,
          dtypes=(torch.float32, torch.float16, torch.bfloat16))
    _need(targets, "targets", (N,), torch.int64, dev)
    if out is None:
        logp = _new((N,), torch.float32, dev, stream)
        lse = _new((N,), torch.float32, dev, stream)
    else:
        logp, lse = out
    _need(logp, "logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    st = L.logits_logp_fwd_ex(_ptr(logits), ld, _code(logits.dtype), _ptr(targets), N, V,
                              _ptr(logp), _ptr(lse), _opts(temperature), _stream(stream))
    _check("logits_logp_fwd", st)
    return logp, lse


def logits_bwd(grad_logp, logits, targets, lse, V=None, *, temperature=1.0, out=None,
               stream=None):
    """grad_logits [N, ld] in the logits dtype (columns [0, V) written)."""
    torch = _torch()
    L = load()
    N, ld = logits.shape
    V = ld if V is None else V
    dev = logits.device
    _need(logits, "logits", (N, ld), device=dev,
          dtypes=(torch.float32, torch.float16, torch.bfloat16))
    _need(targets, "targets", (N,), torch.int64, dev)
    _need(grad_logp, "grad_logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    if out is None:
        out = _new((N, ld), logits.dtype, dev, stream)
    _need(out, "grad_logits", (N, ld), logits.dtype, dev)
    st = L.logits_logp_bwd_ex(_ptr(grad_logp), _ptr(logits), ld, _code(logits.dtype),
                              _ptr(targets), _ptr(lse), N, V, _ptr(out), _opts(temperature),
                              _stream(stream))
    _check("logits_logp_bwd", st)
    return out


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(load().ll_launch_count())


def profile(enable: bool):
    """Start (clearing earlier records) or stop per-phase CUDA-event tracing."""
    load().ll_profile_enable(int(bool(enable)))


def profile_summary() -> dict:
    """{phase: (count, total_ms)} of the recorded phases (synchronises)."""
    buf = ctypes.create_string_buffer(8192)
    n = load().ll_profile_summary(buf, len(buf))
    if n < 0:
        raise LLError("ll_profile_summary", -n)
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, ms = line.split()
        out[name] = (int(cnt), float(ms))
    return out


def logits_fwd_bwd(grad_logp, logits, targets, V=None, *, temperature=1.0, out=None,
                   stream=None):
    """(logp, lse, grad_logits) in one pass over the logits (grad_logp known
    before the forward)."""
    torch = _torch()
    L = load()
    N, ld = logits.shape
    V = ld if V is None else V
    dev = logits.device
    _need(logits, "logits", (N, ld), device=dev,
          dtypes=(torch.float32, torch.float16, torch.bfloat16))
    _need(targets, "targets", (N,), torch.int64, dev)
    _need(grad_logp, "grad_logp", (N,), torch.float32, dev)
    if out is None:
        logp = _new((N,), torch.float32, dev, stream)
        lse = _new((N,), torch.float32, dev, stream)
        g = _new((N, ld), logits.dtype, dev, stream)
    else:
        logp, lse, g = out
    _need(logp, "logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    _need(g, "grad_logits", (N, ld), logits.dtype, dev)
    st = L.logits_logp_fwd_bwd_ex(_ptr(grad_logp), _ptr(logits), ld, _code(logits.dtype),
                                  _ptr(targets), N, V, _ptr(logp), _ptr(lse), _ptr(g),
                                  _opts(temperature), _stream(stream))
    _check("logits_logp_fwd_bwd", st)
    return logp, lse, g


def sum_ordered(parts, out=None, stream=None):
    """out[i] = parts[0, i] + parts[1, i] + ... in ascending order (FP32
    accumulation, one rounding to the dtype): parts is a device tensor
    [nparts, n] (contiguous rows), out [n]."""
    torch = _torch()
    L = load()
    if parts.dim() != 2 or not parts.is_cuda or parts.stride(1) != 1:
        raise ValueError("parts must be a CUDA tensor [nparts, n] with contiguous rows")
    k, n = parts.shape
    if out is None:
        out = _new((n,), parts.dtype, parts.device, stream)
    _need(out, "out", (n,), parts.dtype, parts.device)
    st = L.ll_sum_ordered(_ptr(parts), k, n, parts.stride(0), _code(parts.dtype), _ptr(out),
                          _stream(stream))
    _check("ll_sum_ordered", st)
    return out


def check_status(stream=None) -> int:
    """Synchronise and return (and clear) the device-side status word."""
    return int(load().ll_check_status(_stream(stream)))


# ---------------------------------------------------------- vocab shards

def shard_segments(Vs: int) -> int:
    """LSE segments of a vocab shard of Vs entries."""
    return int(load().ll_shard_segments(int(Vs)))


def forward_shard(hidden, weight, bias, targets, v0, V, *, temperature=1.0, workspace=None,
                  out=None, stream=None):
    """Segment partials of the vocab shard [v0, v0 + weight.shape[0]) of a
    vocab of V entries: (part_m, part_s) [shard_segments(Vs), N] and zy [N]
    (z of the target where it lies in the shard, -inf elsewhere).  targets
    are global ids."""
    torch = _torch()
    L = load()
    N, D, Vs, dev = _check_linear(hidden, weight, bias, targets)
    code = _code(hidden.dtype)
    S = shard_segments(Vs)
    if out is None:
        part_m = _new((S, N), torch.float32, dev, stream)
        part_s = _new((S, N), torch.float32, dev, stream)
        zy = _new((N,), torch.float32, dev, stream)
    else:
        part_m, part_s, zy = out
    _need(part_m, "part_m", (S, N), torch.float32, dev)
    _need(part_s, "part_s", (S, N), torch.float32, dev)
    _need(zy, "zy", (N,), torch.float32, dev)
    if workspace is None:
        workspace = _workspace(L.ll_workspace_size_shard(N, D, Vs, code, 0, 0, 0), dev,
                               stream)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    st = L.ll_forward_shard(_ptr(hidden), _ptr(weight), _ptr(bias), _ptr(targets), N, D, Vs,
                            int(v0), int(V), code, _ptr(part_m), _ptr(part_s), _ptr(zy),
                            _ptr(workspace), workspace.numel(), _opts(temperature),
                            _stream(stream))
    _check("ll_forward_shard", st)
    return part_m, part_s, zy


def lse_merge(part_m, part_s, zy, targets, V, *, out=None, stream=None):
    """(logp, lse) from whole-vocab segment partials [n_segs, N] in ascending
    segment order (rows of m = -inf, s = 0 change nothing)."""
    torch = _torch()
    L = load()
    if part_m.dim() != 2:
        raise ValueError("part_m must be 2-D [n_segs, N]")
    n_segs, N = part_m.shape
    dev = part_m.device
    _need(part_m, "part_m", (n_segs, N), torch.float32, dev)
    _need(part_s, "part_s", (n_segs, N), torch.float32, dev)
    _need(zy, "zy", (N,), torch.float32, dev)
    _need(targets, "targets", (N,), torch.int64, dev)
    if out is None:
        logp = _new((N,), torch.float32, dev, stream)
        lse = _new((N,), torch.float32, dev, stream)
    else:
        logp, lse = out
    _need(logp, "logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    st = L.ll_lse_merge(_ptr(part_m), _ptr(part_s), n_segs, N, _ptr(zy), _ptr(targets), N,
                        int(V), _ptr(logp), _ptr(lse), _stream(stream))
    _check("ll_lse_merge", st)
    return logp, lse


def backward_shard(grad_logp, hidden, weight, bias, targets, lse, v0, V, *, need_dh=True,
                   need_dw=True, need_db=None, dh_dtype=None, dw_dtype=None, token_chunks=0,
                   temperature=1.0, split_s="auto", workspace=None, out=None, stream=None):
    """(grad_hidden part, grad_weight rows, grad_bias rows) of the vocab shard
    [v0, v0 + weight.shape[0]); lse is the merged whole-vocab lse.  The
    grad_hidden part defaults to float32 (the shards' parts are summed)."""
    torch = _torch()
    L = load()
    N, D, Vs, dev = _check_linear(hidden, weight, bias, targets)
    code = _code(hidden.dtype)
    if need_db is None:
        need_db = bias is not None
    if dh_dtype is None and (out is None or out[0] is None):
        dh_dtype = torch.float32
    _need(grad_logp, "grad_logp", (N,), torch.float32, dev)
    _need(lse, "lse", (N,), torch.float32, dev)
    dh, dW, db, dh_dtype, dw_dtype = _grad_outputs(out, need_dh, need_dw, need_db, N, D, Vs,
                                                   hidden.dtype, dh_dtype, dw_dtype, dev,
                                                   stream)
    if workspace is None:
        workspace = _workspace(L.ll_workspace_size_shard(
            N, D, Vs, code, token_chunks, 1, int(bool(need_db)) | (_split_code(split_s) << 1)),
            dev, stream)
    _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    st = L.ll_backward_shard(_ptr(grad_logp), _ptr(hidden), _ptr(weight), _ptr(bias),
                             _ptr(targets), _ptr(lse), N, D, Vs, int(v0), int(V), code,
                             int(bool(need_dh)), int(bool(need_dw)), int(bool(need_db)),
                             _ptr(dh), _code(dh_dtype), _ptr(dW), _code(dw_dtype), _ptr(db),
                             int(token_chunks), _ptr(workspace), workspace.numel(),
                             _opts(temperature, split_s), _stream(stream))
    _check("ll_backward_shard", st)
    return dh, dW, db


# ------------------------------------------------- the rest of a training step
# Calls of a few microseconds: pointers go to ctypes as plain integers, and the
# checks build nothing unless they fail.

def _rows(t, name):
    """(rows, columns, row stride) of a 2-D tensor whose rows are contiguous."""
    codes = _CODES or _codes()
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.dtype not in codes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {tuple(codes)}")
    n, d = t.shape
    if t.is_contiguous():
        return n, d, d
    ld, one = t.stride()
    if n <= 1:
        ld = d
    if (d > 1 and one != 1) or ld < d:
        raise ValueError(f"{name}: each row must be contiguous and the rows apart")
    return n, d, ld


def _vector(t, name, n, dtype, device):
    """Raise unless t is a contiguous [n] tensor of `dtype` on `device`."""
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 1 and
            t.shape[0] == n and t.device == device and t.is_contiguous()):
        _need(t, name, (n,), dtype, device)


_CODES: dict = {}


def _codes():
    """torch dtype -> ll_dtype code."""
    if not _CODES:
        _CODES.update(DTYPE_CODES())
    return _CODES


def _stream_of(device, stream):
    """The stream of a call whose tensors lie on `device`, as a handle."""
    if stream is not None:
        return stream.cuda_stream
    if device.type != "cuda":
        return None  # the call itself then fails: no device memory
    # a name of torch's own, which other versions may lack: it saves the Stream object
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw else _torch().cuda.current_stream(device).cuda_stream


def _scratch(workspace, nbytes, device, stream):
    """The given workspace, checked, or a new one."""
    torch = _torch()
    if workspace is None:
        return _new((max(nbytes, 256),), torch.uint8, device, stream, scratch=True)
    _vector(workspace, "workspace", workspace.numel(), torch.uint8, device)
    return workspace


def embed_forward(weight, tokens, *, scale=1.0, v0=0, out_dtype=None, out=None, stream=None):
    """out [N, D] = scale * weight[tokens - v0], +0 rows for tokens outside
    [v0, v0 + V).  weight [V, D] and out may have a row stride.  out_dtype
    defaults to weight's; FP32 is always possible, and anything from FP32."""
    torch = _torch()
    L = load()
    codes = _codes()
    V, D, ldw = _rows(weight, "weight")
    dev = weight.device
    N = tokens.shape[0] if isinstance(tokens, torch.Tensor) and tokens.dim() else 0
    _vector(tokens, "tokens", N, torch.int64, dev)
    if out is None:
        if out_dtype is None:
            out_dtype = weight.dtype
        elif out_dtype not in codes:
            raise TypeError(f"out_dtype {out_dtype}, expected one of {tuple(codes)}")
        out, ldo = _new((N, D), out_dtype, dev, stream), D
    else:
        if out_dtype is not None and out_dtype != out.dtype:
            raise TypeError("out_dtype disagrees with the given out")
        n, d, ldo = _rows(out, "out")
        if n != N or d != D or out.device != dev:
            raise ValueError(f"out: {(n, d)} on {out.device}, expected {(N, D)} on {dev}")
    st = L.ll_embed_forward(weight.data_ptr(), ldw, codes[weight.dtype], tokens.data_ptr(), N, D,
                            V, v0, scale, out.data_ptr(), ldo, codes[out.dtype],
                            _stream_of(dev, stream))
    if st:
        raise LLError("ll_embed_forward", st)
    return out


def embed_backward(grad_out, tokens, V, *, scale=1.0, v0=0, dw_dtype=None, accumulate=False,
                   out=None, workspace=None, stream=None):
    """grad_weight [V, D] of embed_forward: row v the sum of scale * grad_out[n]
    over the n with tokens[n] == v0 + v.  dw_dtype (FP32 by default, or
    grad_out's) is that of `out` when given.  accumulate=True adds into `out`
    (tied weights: the grad_weight of `backward`)."""
    torch = _torch()
    L = load()
    codes = _codes()
    N, D, ldg = _rows(grad_out, "grad_out")
    V = int(V)
    dev = grad_out.device
    _vector(tokens, "tokens", N, torch.int64, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the table to add into (out)")
        if dw_dtype is None:
            dw_dtype = torch.float32
        elif dw_dtype not in codes:
            raise TypeError(f"dw_dtype {dw_dtype}, expected one of {tuple(codes)}")
        out, ldw = _new((V, D), dw_dtype, dev, stream), D
    else:
        if dw_dtype is not None and dw_dtype != out.dtype:
            raise TypeError("dw_dtype disagrees with the given out")
        v, d, ldw = _rows(out, "out")
        if v != V or d != D or out.device != dev:
            raise ValueError(f"out: {(v, d)} on {out.device}, expected {(V, D)} on {dev}")
    workspace = _scratch(workspace, L.ll_embed_workspace_size(N, D, V), dev, stream)
    st = L.ll_embed_backward(grad_out.data_ptr(), ldg, codes[grad_out.dtype], tokens.data_ptr(), N,
                             D, V, v0, scale, 1 if accumulate else 0, out.data_ptr(), ldw,
                             codes[out.dtype], workspace.data_ptr(), workspace.shape[0],
                             _stream_of(dev, stream))
    if st:
        raise LLError("ll_embed_backward", st)
    return out


class PolicyOptions(ctypes.Structure):
    """ll_policy_options of the C ABI."""
    _fields_ = [("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double),
                ("kl_coef", ctypes.c_double), ("denominator", ctypes.c_double),
                ("reserved", ctypes.c_int * 4)]


def policy_loss(logp, old_logp, advantages, *, ref_logp=None, mask=None, seq_offsets=None,
                clip_low=0.2, clip_high=0.2, kl_coef=0.0, denominator=None, out=None,
                workspace=None, stream=None):
    """(stats [4], grad_logp [N]), FP32, of the clipped policy loss: stats are
    the loss, its policy part, the divergence from ref_logp and the clipped
    share; grad_logp is what `backward` takes.

    mask [N] (bool or uint8): tokens that count.  The loss is the mean over
    them, or with seq_offsets ([B + 1] int64, on the device) the mean over the
    sequences of each sequence's mean; denominator replaces the number of
    tokens (sequences) of this call."""
    torch = _torch()
    L = load()
    f32 = torch.float32
    if not isinstance(logp, torch.Tensor) or logp.dim() != 1:
        raise TypeError("logp must be a 1-D torch.Tensor")
    N, dev = logp.shape[0], logp.device
    _vector(logp, "logp", N, f32, dev)
    _vector(old_logp, "old_logp", N, f32, dev)
    _vector(advantages, "advantages", N, f32, dev)
    ref = msk = offs = None
    B = 0
    if ref_logp is not None:
        _vector(ref_logp, "ref_logp", N, f32, dev)
        ref = ref_logp.data_ptr()
    if mask is not None:
        _need(mask, "mask", (N,), device=dev, dtypes=(torch.bool, torch.uint8))
        msk = mask.data_ptr()
    if seq_offsets is not None:
        B = seq_offsets.numel() - 1 if isinstance(seq_offsets, torch.Tensor) else 0
        _vector(seq_offsets, "seq_offsets", B + 1, torch.int64, dev)
        if B < 1:
            raise ValueError("seq_offsets: at least two are needed")
        offs = seq_offsets.data_ptr()
    if denominator is None:
        denominator = 0.0
    elif not denominator > 0:
        raise ValueError("denominator must be > 0")
    if out is None:
        stats, grad = _new((4,), f32, dev, stream), _new((N,), f32, dev, stream)
    else:
        stats, grad = out
        _vector(stats, "stats", 4, f32, dev)
        _vector(grad, "grad_logp", N, f32, dev)
    workspace = _scratch(workspace, L.ll_policy_workspace_size(N, B), dev, stream)
    opt = PolicyOptions(clip_low, clip_high, kl_coef, denominator)
    st = L.ll_policy_loss(logp.data_ptr(), old_logp.data_ptr(), ref, advantages.data_ptr(), msk,
                          offs, B, N, ctypes.byref(opt), stats.data_ptr(), grad.data_ptr(),
                          workspace.data_ptr(), workspace.shape[0], _stream_of(dev, stream))
    if st:
        raise LLError("ll_policy_loss", st)
    return stats, grad


class Tensor(ctypes.Structure):
    """ll_tensor of the C ABI."""
    _fields_ = [("data", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("reserved", ctypes.c_int)]


def _tensor_list(tensors):
    """(ll_tensor records as three 64-bit integers each, device) of gradients
    that each fill their memory without gaps, in any order of their dimensions."""
    T = _torch().Tensor
    codes = _codes()
    if not isinstance(tensors, (list, tuple)):
        tensors = list(tensors)
    words = array.array("q", bytes(24 * len(tensors)))  # the dtype shares its word with reserved = 0
    try:
        words[0::3] = array.array("q", map(T.data_ptr, tensors))
        words[1::3] = array.array("q", map(T.numel, tensors))
        words[2::3] = array.array("q", [codes[t.dtype] for t in tensors])
        alike = len(set(map(T.get_device, tensors))) <= 1 and all(map(T.is_contiguous, tensors))
    except (TypeError, KeyError):
        alike = False
    if not alike:
        for i, t in enumerate(tensors):
            if not isinstance(t, T):
                raise TypeError(f"tensor {i} must be a torch.Tensor")
            if t.dtype not in codes:
                raise TypeError(f"tensor {i}: unsupported dtype {t.dtype}")
            if t.device != tensors[0].device:
                raise ValueError(f"tensor {i}: on {t.device}, expected {tensors[0].device}")
            if not t.is_contiguous() and not _dense(t):
                raise ValueError(f"tensor {i}: its elements must fill their memory without gaps")
    return words, tensors[0].device if tensors else None


def _dense(t):
    """Whether some order of the dimensions makes the tensor contiguous."""
    need = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != need:
            return False
        need *= size
    return True


def _norm_call(tensors, norm, workspace, stream):
    torch = _torch()
    L = load()
    words, dev = _tensor_list(tensors)
    if dev is None:
        dev = norm.device if norm is not None else torch.device("cuda", torch.cuda.current_device())
    if norm is None:
        norm = _new((), torch.float32, dev, stream)
    else:
        _need(norm, "norm", (), torch.float32, dev)
    count = len(words) // 3
    workspace = _scratch(workspace, L.ll_grad_norm_workspace_size(count), dev, stream)
    return L, words, count, dev, norm, workspace


def grad_norm(tensors, *, out=None, workspace=None, stream=None):
    """The norm (0-d FP32) of a list of gradients taken as one vector.  Their
    dtypes may differ; each must fill its memory without gaps."""
    L, words, count, dev, out, workspace = _norm_call(tensors, out, workspace, stream)
    st = L.ll_grad_norm(words.buffer_info()[0], count, out.data_ptr(), workspace.data_ptr(),
                        workspace.shape[0], _stream_of(dev, stream))
    if st:
        raise LLError("ll_grad_norm", st)
    return out


def clip_grads(tensors, max_norm, *, norm=None, workspace=None, stream=None):
    """Scales a list of gradients in place by min(1, max_norm / (norm + 1e-6))
    and returns norm: that of the list, or a given one (0-d FP32 on the device:
    gradients sharded over ranks)."""
    given = norm is not None
    L, words, count, dev, norm, workspace = _norm_call(tensors, norm, workspace, stream)
    st = L.ll_clip_grads(words.buffer_info()[0], count, max_norm, 1 if given else 0,
                         norm.data_ptr(), workspace.data_ptr(), workspace.shape[0],
                         _stream_of(dev, stream))
    if st:
        raise LLError("ll_clip_grads", st)
    return norm


# ------------------------------------------- the rollout side of the vocabulary

FP4_FORMATS = {"mx": 0, "nv": 1}


class FP4Matrix:
    """A matrix [rows, cols] in microscaled 4-bit floating point, as the C ABI
    lays it out: `codes` [rows, bytes of a row] uint8, `scales` uint8 (tiles of
    128 rows x 4 blocks) and, for format "nv", `scale` (one FP32 on the device;
    None for "mx")."""
    __slots__ = ("codes", "scales", "scale", "cols", "format")

    def __init__(self, codes, scales, scale, cols, format="mx"):
        torch = _torch()
        if format not in FP4_FORMATS:
            raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}")
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise TypeError("codes must be a 2-D torch.Tensor")
        L = load()
        cols = int(cols)
        rows, dev, u8 = codes.shape[0], codes.device, torch.uint8
        _need(codes, "codes", (rows, L.ll_fp4_row_bytes(cols)), u8, dev)
        _need(scales, "scales", (L.ll_fp4_scale_bytes(rows, cols, FP4_FORMATS[format]),), u8, dev)
        if (format == "nv") != (scale is not None):
            raise ValueError('scale belongs to format "nv"')
        if scale is not None:
            _need(scale, "scale", (), torch.float32, dev)
        self.codes, self.scales, self.scale = codes, scales, scale
        self.cols, self.format = cols, format

    @property
    def shape(self):
        return self.codes.shape[0], self.cols

    @property
    def device(self):
        return self.codes.device

    def _ptrs(self):
        return (self.codes.data_ptr(), self.scales.data_ptr(),
                None if self.scale is None else self.scale.data_ptr())


def _fp4(codes, scales, scale, cols, format):
    """An FP4Matrix of buffers that need no check."""
    q = FP4Matrix.__new__(FP4Matrix)
    q.codes, q.scales, q.scale, q.cols, q.format = codes, scales, scale, cols, format
    return q


def _is_fp4(q, name):
    if not isinstance(q, FP4Matrix):
        raise TypeError(f"{name} must be an FP4Matrix (of fp4_quantize)")


def fp4_quantize(x, format="mx", *, scale=None, out=None, stream=None):
    """FP4Matrix of x [R, K] (FP32, FP16 or BF16, rows may have a stride).
    "mx": blocks of 32 columns with power-of-two scales; "nv": blocks of 16 with
    E4M3 scales, relative to `scale`: a 0-d FP32 on the device that the user
    keeps (a calibrated activation scale), or None: computed from x and kept in
    the result.  out: an FP4Matrix of the same shape and format to write (without
    `scale` its scale is written too, also one that it was made with)."""
    torch = _torch()
    L = _LIB or load()
    code = FP4_FORMATS.get(format)
    if code is None:
        raise ValueError(f"format must be one of {sorted(FP4_FORMATS)}")
    R, K, ldx = _rows(x, "x")
    dev = x.device
    if K < 1:
        raise ValueError("x: at least one column is needed")
    given = scale is not None
    if given:
        if not code:
            raise ValueError('scale belongs to format "nv"')
        if not (isinstance(scale, torch.Tensor) and scale.dtype is torch.float32 and
                not scale.dim() and scale.device == dev):
            _need(scale, "scale", (), torch.float32, dev)
    if out is None:
        u8 = torch.uint8
        if code and not given:
            scale = _new((), torch.float32, dev, stream)
        # what ll_fp4_row_bytes and ll_fp4_scale_bytes give
        tile = 64 if code else 128
        n = (R + 127) // 128 * ((K + tile - 1) // tile) * 512
        out = _fp4(_new((R, (K + 31) // 32 * 16), u8, dev, stream), _new((n,), u8, dev, stream),
                   scale, K, format)
    else:
        _is_fp4(out, "out")
        if out.shape != (R, K) or out.format != format or out.device != dev:
            raise ValueError(f"out: {out.shape} {out.format!r} on {out.device}, expected "
                             f"{(R, K)} {format!r} on {dev}")
        if given:
            out = _fp4(out.codes, out.scales, scale, K, format)
    codes, scales, g = out._ptrs()
    st = L.ll_fp4_quantize(x.data_ptr(), ldx, _codes()[x.dtype], R, K, code, g, 1 if given else 0,
                           codes, scales, _stream_of(dev, stream))
    if st:
        raise LLError("ll_fp4_quantize", st)
    return out


def _out_2d(out, out_dtype, default, shape, dev, stream):
    """(out, row stride) of a call that writes a 2-D tensor: the given one,
    checked, or a new one of out_dtype."""
    if out is None:
        if out_dtype is None:
            out_dtype = default
        elif out_dtype not in (_CODES or _codes()):
            raise TypeError(f"out_dtype {out_dtype}, expected one of {tuple(_codes())}")
        return _new(shape, out_dtype, dev, stream), shape[1]
    if out_dtype is not None and out_dtype != out.dtype:
        raise TypeError("out_dtype disagrees with the given out")
    n, d, ldo = _rows(out, "out")
    if (n, d) != shape or out.device != dev:
        raise ValueError(f"out: {(n, d)} on {out.device}, expected {shape} on {dev}")
    return out, ldo


def fp4_dequantize(q, out_dtype=None, *, out=None, stream=None):
    """The values that an FP4Matrix stands for, [R, K] in out_dtype (FP32 by
    default)."""
    L = _LIB or load()
    if not isinstance(q, FP4Matrix):
        _is_fp4(q, "q")
    codes, K = q.codes, q.cols
    R, dev = codes.shape[0], codes.device
    out, ldo = _out_2d(out, out_dtype, _torch().float32, (R, K), dev, stream)
    scale = q.scale
    st = L.ll_fp4_dequantize(codes.data_ptr(), q.scales.data_ptr(),
                             None if scale is None else scale.data_ptr(), R, K,
                             FP4_FORMATS[q.format], out.data_ptr(), ldo, _codes()[out.dtype],
                             _stream_of(dev, stream))
    if st:
        raise LLError("ll_fp4_dequantize", st)
    return out


def fp4_linear(hidden, weight, bias=None, *, out_dtype=None, out=None, stream=None):
    """Logits [N, V] = hidden . weight^T (+ bias) of two FP4Matrix of one format,
    [N, K] and [V, K], in out_dtype (BF16 by default): what `sample` and
    `logits_fwd` take.  bias [V] in FP32, FP16 or BF16."""
    torch = _torch()
    L = _LIB or load()
    _is_fp4(hidden, "hidden")
    _is_fp4(weight, "weight")
    (N, K), V, dev = hidden.shape, weight.shape[0], hidden.device
    if weight.cols != K or weight.format != hidden.format or weight.device != dev:
        raise ValueError(f"weight: {weight.cols} columns of format {weight.format!r} on "
                         f"{weight.device}, expected {K} of {hidden.format!r} on {dev}")
    if V < 1:
        raise ValueError("weight: at least one row is needed")
    b, b_code = None, 0
    if bias is not None:
        _need(bias, "bias", (V,), device=dev, dtypes=tuple(_codes()))
        b, b_code = bias.data_ptr(), _codes()[bias.dtype]
    out, ldo = _out_2d(out, out_dtype, torch.bfloat16, (N, V), dev, stream)
    st = L.ll_fp4_linear(*hidden._ptrs(), *weight._ptrs(), b, b_code, N, K, V,
                         FP4_FORMATS[hidden.format], out.data_ptr(), ldo, _codes()[out.dtype],
                         _stream_of(dev, stream))
    if st:
        raise LLError("ll_fp4_linear", st)
    return out


class SampleOptions(ctypes.Structure):
    """ll_sample_options of the C ABI."""
    _fields_ = [("temperature", ctypes.c_double), ("top_p", ctypes.c_double),
                ("min_p", ctypes.c_double), ("top_k", ctypes.c_int64),
                ("temperatures", ctypes.c_void_p), ("top_ps", ctypes.c_void_p),
                ("min_ps", ctypes.c_void_p), ("top_ks", ctypes.c_void_p),
                ("reserved", ctypes.c_int * 4)]


def sample(logits, uniforms, V=None, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None,
           workspace=None, stream=None):
    """(tokens [N] int64, logp [N], logq [N] FP32): one token drawn from each row
    of logits [N, ld] (rows may have a stride; columns >= V, default all,
    ignored) by its random number of uniforms [N] (FP32, in [0, 1)).

    temperature (0: the likeliest token), top_k (0: off), top_p (1: off) and
    min_p (0: off) are numbers, or tensors [N] on the device (FP32; top_k
    int32) that give each row its own.  logp is the token's log-probability at
    this temperature before anything is cut off (the old_logp of policy_loss,
    the logp of logits_fwd), logq the one it was drawn with.  A row without a
    finite logit gives token -1 and zeros."""
    torch = _torch()
    L = _LIB or load()
    N, cols, ld = _rows(logits, "logits")
    V = cols if V is None else int(V)
    if not 1 <= V <= cols:
        raise ValueError(f"V: {V}, expected 1 to {cols}")
    dev, f32 = logits.device, torch.float32
    _vector(uniforms, "uniforms", N, f32, dev)
    Tensor = torch.Tensor
    if (isinstance(temperature, Tensor) or isinstance(top_k, Tensor) or
            isinstance(top_p, Tensor) or isinstance(min_p, Tensor)):
        opt = SampleOptions()
        for name, v, dtype in (("temperature", temperature, f32), ("top_p", top_p, f32),
                               ("min_p", min_p, f32), ("top_k", top_k, torch.int32)):
            if isinstance(v, Tensor):
                _vector(v, name, N, dtype, dev)
                setattr(opt, name + "s", v.data_ptr())
            else:
                setattr(opt, name, v)
    else:
        opt = SampleOptions(temperature, top_p, min_p, top_k)
    if out is None:
        tokens = _new((N,), torch.int64, dev, stream)
        logp, logq = _new((N,), f32, dev, stream), _new((N,), f32, dev, stream)
    else:
        tokens, logp, logq = out
        _vector(tokens, "tokens", N, torch.int64, dev)
        _vector(logp, "logp", N, f32, dev)
        _vector(logq, "logq", N, f32, dev)
    code = _CODES[logits.dtype]
    workspace = _scratch(workspace, L.ll_sample_workspace_size(N, V, code), dev, stream)
    st = L.ll_sample(logits.data_ptr(), ld, code, uniforms.data_ptr(), N, V, ctypes.byref(opt),
                     tokens.data_ptr(), logp.data_ptr(), logq.data_ptr(), workspace.data_ptr(),
                     workspace.shape[0], _stream_of(dev, stream))
    if st:
        raise LLError("ll_sample", st)
    return tokens, logp, logq
