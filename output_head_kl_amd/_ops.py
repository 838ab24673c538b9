"""The operators beside the loss: log probabilities of given tokens (from logits and from
hidden states) with their gradients, and the gradient norm with clipping.  Thin, as the rest
of the binding: arguments are checked, outputs and workspaces allocated with torch, and the
library's HIP kernels do the work on the current stream (or on ``stream``).  No call
synchronises, so each can be recorded with ``torch.cuda.graph``."""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools
import operator

import torch

import output_head_kl_amd as kd

_F32 = torch.float32
_CODES = {torch.bfloat16: kd.KD_BF16, _F32: kd.KD_F32}


def declare(lib) -> None:
    """Argument types of the operators' C calls."""
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
    psz = ctypes.POINTER(sz)
    for name, args in (
            ("kd_token_logprobs_workspace_bytes", [i64, i64, i32, i32, psz]),
            ("kd_token_logprobs", [vp, i32, i64, vp, i32, i64, i64, i32, vp, vp, vp, vp, vp, vp,
                                   vp, vp, sz, vp]),
            ("kd_token_logprobs_bwd", [vp, i32, i64, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp,
                                       i64, vp]),
            ("kd_head_logprobs_workspace_bytes", [i64, i64, i64, i64, i32, psz]),
            ("kd_head_logprobs", [vp, vp, i32, vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp,
                                  vp, sz, vp]),
            ("kd_head_logprobs_bwd_workspace_bytes", [i64, i64, i64, i64, i32, i32, i64, psz]),
            ("kd_head_logprobs_bwd", [vp, vp, i32, vp, i32, i64, i64, i64, i64, vp, vp, vp, vp,
                                      vp, vp, vp, i32, vp, sz, vp]),
            ("kd_clip_grads_workspace_bytes", [vp, i32, psz]),
            ("kd_clip_grads", [vp, vp, vp, vp, i32, ctypes.c_float, vp, vp, sz, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int


@contextlib.contextmanager
def _on(dev, stream):
    """The call's device and stream as torch's current ones, so that what the call allocates
    belongs to the stream that uses it."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            with torch.cuda.stream(stream):
                yield


def _raw_stream(dev):
    """The handle of torch's current stream on dev (by the short way where torch has it)."""
    return _CURRENT(dev.index) if _CURRENT else torch.cuda.current_stream(dev).cuda_stream


_CURRENT = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _elsewhere(dev, stream) -> bool:
    """Whether the call needs ``_on``: another stream or another device than the current."""
    return stream is not None or torch.cuda.current_device() != dev.index


def _rows(t, name):
    """(N, V, elements between rows) of a 2-D tensor whose rows are contiguous and apart."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, not {t.dim()}-D")
    N, V = t.shape
    if V < 1 or (V > 1 and t.stride(1) != 1) or (N > 1 and t.stride(0) < V):
        raise ValueError(f"{name} must have contiguous rows that do not overlap "
                         f"(shape {tuple(t.shape)}, strides {t.stride()})")
    return N, V, t.stride(0) if N > 1 else V


def _token_bits(tokens, N):
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"tokens must be int32 or int64, not {tokens.dtype}")
    if tokens.dim() != 1 or tokens.shape[0] != N or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous tensor of shape [{N}]")
    return 64 if tokens.dtype == torch.int64 else 32


def _status_ptr(status):
    if status is None:
        return None
    if status.dtype != torch.int32 or status.numel() != 1:
        raise ValueError("status must be a one-element int32 tensor")
    return status.data_ptr()


def _upstream(name, g, N, dev):
    """An upstream gradient as the library reads it: None, or contiguous float32 [N]."""
    if g is None:
        return None
    kd._on_device(dev, **{name: g})
    if tuple(g.shape) != (N,):
        raise ValueError(f"{name} must have shape [{N}]")
    return g.to(_F32).contiguous()


def _float_rows(name, t, shape):
    if t.dtype != _F32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {list(shape)}")


def _scratch(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    kd._check_workspace(workspace, dev)
    return workspace


@functools.lru_cache(maxsize=1024)
def token_logprobs_workspace_bytes(N: int, V: int, top: int = 0, dtype: int = kd.KD_BF16) -> int:
    """Workspace bytes of ``token_logprobs`` (0 for many rows)."""
    out = ctypes.c_size_t(0)
    kd._check(kd._lib().kd_token_logprobs_workspace_bytes(N, V, top, dtype, ctypes.byref(out)))
    return int(out.value)


def _code(t, name):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}") from None


def _same_device(dev, **tensors):
    """kd._on_device without its message unless there is one to give."""
    for t in tensors.values():
        if t is not None and t.device != dev:
            kd._on_device(dev, **tensors)


def _token_logprobs(logits, tokens, top, status, workspace, stats):
    dt = _code(logits, "logits")
    dev = logits.device
    _same_device(dev, tokens=tokens, status=status)
    N, V, ld = _rows(logits, "logits")
    if not 0 <= top <= V:
        raise ValueError(f"top = {top} outside [0, {V}]")
    bits = _token_bits(tokens, N)
    workspace = _scratch(workspace, token_logprobs_workspace_bytes(N, V, top, dt), dev)
    logp = torch.empty(N, dtype=_F32, device=dev)
    entropy = torch.empty(N, dtype=_F32, device=dev)
    lse = torch.empty(N, dtype=_F32, device=dev)
    st = torch.empty((N, 2), dtype=_F32, device=dev) if stats else None
    idx = torch.empty((N, top), dtype=torch.int32, device=dev) if top else None
    tlp = torch.empty((N, top), dtype=_F32, device=dev) if top else None
    kd._check(kd._lib().kd_token_logprobs(
        logits.data_ptr(), dt, ld, tokens.data_ptr(), bits, N, V, top, logp.data_ptr(),
        entropy.data_ptr(), lse.data_ptr(), kd._ptr(st), kd._ptr(idx), kd._ptr(tlp),
        _status_ptr(status), kd._ptr(workspace), 0 if workspace is None else workspace.numel(),
        _raw_stream(dev)))
    return (logp, entropy, lse, idx, tlp) if top else (logp, entropy, lse), st


def token_logprobs(logits, tokens, top: int = 0, status=None, workspace=None, stream=None):
    """Log probabilities of given tokens from logits, with entropy and top alternatives.

    Args (torch CUDA tensors):
      logits [N, V]: bfloat16 or float32, rows contiguous (any distance between rows);
      tokens [N]: int32 or int64, negative where a row has no token.
      top: number of alternatives, 0 to 64.
      status: optional int32 tensor of one element, set to 2 (KD_E_INDEX) when a token is
        not below V or a row holds NaN or +inf (never cleared).
      workspace: optional uint8 tensor of ``token_logprobs_workspace_bytes`` bytes.
      stream: a torch.cuda.Stream or a raw handle; the current stream by default.
    Returns (logp [N], entropy [N], lse [N]) float32 and, with ``top``, (top_idx [N, top]
    int32, top_logp [N, top] float32), the largest logits first, equal ones by rising index.
    logp is 0 without a token; a row with no finite logit has logp = lse = -inf, entropy 0; an
    invalid row NaN.  logp, entropy and lse are differentiable in logits (the alternatives are
    not); the backward reads logits again.  Before a backward is captured into a graph, drop
    eager results of the same leaf (or detach it): torch fails on their streams otherwise."""
    dev = logits.device
    kd._on_device(dev, logits=logits)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return token_logprobs(logits, tokens, top, status, workspace)
    if torch.is_grad_enabled() and logits.requires_grad:
        return _TokenLogprobs.apply(logits, tokens, top, status, workspace)
    return _token_logprobs(logits, tokens, top, status, workspace, False)[0]


def token_logprobs_bwd(logits, tokens, row_stats, entropy, grad_logp=None, grad_entropy=None,
                       grad_lse=None, out=None, stream=None):
    """The gradient of the logits (kd_token_logprobs_bwd) for upstream gradients [N] of logp,
    entropy and lse (None: 0).  ``row_stats`` [N, 2] and ``entropy`` [N] come from the
    forward; ``out`` may be given, and may be ``logits`` itself."""
    dev = logits.device
    kd._on_device(dev, logits=logits, tokens=tokens, row_stats=row_stats, entropy=entropy, out=out)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return token_logprobs_bwd(logits, tokens, row_stats, entropy, grad_logp,
                                      grad_entropy, grad_lse, out)
    dt = _code(logits, "logits")
    N, V, ld = _rows(logits, "logits")
    bits = _token_bits(tokens, N)
    _float_rows("row_stats", row_stats, (N, 2))
    _float_rows("entropy", entropy, (N,))
    g = [_upstream(n, x, N, dev) for n, x in (("grad_logp", grad_logp),
                                              ("grad_entropy", grad_entropy),
                                              ("grad_lse", grad_lse))]
    if out is None:
        out = torch.empty((N, V), dtype=logits.dtype, device=dev)
    if out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError("out must have the shape and dtype of logits")
    ld_d = _rows(out, "out")[2]
    kd._check(kd._lib().kd_token_logprobs_bwd(
        logits.data_ptr(), dt, ld, tokens.data_ptr(), bits, N, V, row_stats.data_ptr(),
        entropy.data_ptr(), kd._ptr(g[0]), kd._ptr(g[1]), kd._ptr(g[2]), out.data_ptr(), ld_d,
        _raw_stream(dev)))
    return out


def _f32(g):
    """An upstream gradient that autograd has checked, as the library reads it."""
    if g is None or (g.dtype is _F32 and g.is_contiguous()):
        return g
    return g.to(_F32).contiguous()


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, status, workspace):
        ctx.set_materialize_grads(False)
        outs, st = _token_logprobs(logits, tokens, top, status, workspace, True)
        ctx.save_for_backward(logits, tokens, outs[1])
        ctx.row_stats = st
        if top:
            ctx.mark_non_differentiable(*outs[3:])
        return outs

    @staticmethod
    def backward(ctx, *grads):
        # the arguments were checked by the forward, so only what autograd gives is looked at;
        # with create_graph the slower wrapper marks the result as differentiable once
        return (_token_backward_once if torch.is_grad_enabled() else _token_backward)(ctx, *grads)


def _token_backward(ctx, g_logp, g_entropy, g_lse, *_):
    logits, tokens, entropy = ctx.saved_tensors
    dev = logits.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _token_backward(ctx, g_logp, g_entropy, g_lse)
    N, V = logits.shape
    g = _f32(g_logp), _f32(g_entropy), _f32(g_lse)
    out = torch.empty((N, V), dtype=logits.dtype, device=dev)
    kd._check(kd._lib().kd_token_logprobs_bwd(
        logits.data_ptr(), _CODES[logits.dtype], logits.stride(0) if N > 1 else V,
        tokens.data_ptr(), 64 if tokens.dtype is torch.int64 else 32, N, V,
        ctx.row_stats.data_ptr(), entropy.data_ptr(), kd._ptr(g[0]), kd._ptr(g[1]),
        kd._ptr(g[2]), out.data_ptr(), V, _raw_stream(dev)))
    return out, None, None, None, None


_token_backward_once = torch.autograd.function.once_differentiable(_token_backward)


# ---- from hidden states ------------------------------------------------------------------
@functools.lru_cache(maxsize=1024)
def head_logprobs_workspace_bytes(N: int, d: int, V: int, chunk: int = 4096,
                                  dtype: int = kd.KD_BF16) -> int:
    """Workspace bytes of ``head_logprobs``."""
    out = ctypes.c_size_t(0)
    kd._check(kd._lib().kd_head_logprobs_workspace_bytes(N, d, V, chunk, dtype, ctypes.byref(out)))
    return int(out.value)


@functools.lru_cache(maxsize=1024)
def head_logprobs_bwd_workspace_bytes(N: int, d: int, V: int, chunk: int = 4096,
                                      dtype: int = kd.KD_BF16, dw_dtype: int = kd.KD_F32,
                                      dw_group_tokens: int = 16384) -> int:
    """Workspace bytes of ``head_logprobs_bwd``: for full speed, or for dW groups of at most
    ``dw_group_tokens`` tokens (0: groups of one chunk)."""
    out = ctypes.c_size_t(0)
    kd._check(kd._lib().kd_head_logprobs_bwd_workspace_bytes(
        N, d, V, chunk, dtype, dw_dtype, dw_group_tokens, ctypes.byref(out)))
    return int(out.value)


def _head(h, W, tokens, **more):
    _same_device(h.device, W=W, tokens=tokens, **more)
    dt = _code(h, "h")
    if W.dtype != h.dtype:
        raise TypeError("h and W must have the same dtype")
    if h.dim() != 2 or W.dim() != 2 or W.shape[1] != h.shape[1]:
        raise ValueError(f"h must be [N, d] and W [V, d], not {tuple(h.shape)}, {tuple(W.shape)}")
    if not h.is_contiguous() or not W.is_contiguous():
        raise ValueError("h and W must be contiguous")
    N, d = h.shape
    return dt, N, d, W.shape[0], _token_bits(tokens, N)


def _head_logprobs(h, W, tokens, chunk, status, workspace, stats):
    dt, N, d, V, bits = _head(h, W, tokens, status=status)
    dev = h.device
    workspace = _scratch(workspace, head_logprobs_workspace_bytes(N, d, V, chunk, dt), dev)
    logp = torch.empty(N, dtype=_F32, device=dev)
    entropy = torch.empty(N, dtype=_F32, device=dev)
    lse = torch.empty(N, dtype=_F32, device=dev)
    st = torch.empty((N, 2), dtype=_F32, device=dev) if stats else None
    kd._check(kd._lib().kd_head_logprobs(
        h.data_ptr(), W.data_ptr(), dt, tokens.data_ptr(), bits, N, d, V, chunk, logp.data_ptr(),
        entropy.data_ptr(), lse.data_ptr(), kd._ptr(st), _status_ptr(status),
        workspace.data_ptr(), workspace.numel(), _raw_stream(dev)))
    return (logp, entropy, lse), st


def head_logprobs(h, W, tokens, chunk: int = 4096, status=None, workspace=None, stream=None):
    """Log probabilities of given tokens from hidden states, with entropy and logsumexp:
    ``token_logprobs`` of h W^T with no logits in memory.

    Args (torch CUDA tensors, contiguous): h [N, d] and W [V, d], bfloat16 or float32 (same
    dtype, d a multiple of 8); tokens [N] int32 or int64, negative where a row has no token;
    chunk: token rows per pass; status, stream: as ``token_logprobs``; workspace: optional
    uint8 tensor of ``head_logprobs_workspace_bytes`` bytes.
    Returns (logp [N], entropy [N], lse [N]) float32, differentiable in h and W: the backward
    recomputes the logits chunk by chunk.  Capturing it: as ``token_logprobs``."""
    dev = h.device
    kd._on_device(dev, h=h)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return head_logprobs(h, W, tokens, chunk, status, workspace)
    if torch.is_grad_enabled() and (h.requires_grad or W.requires_grad):
        return _HeadLogprobs.apply(h, W, tokens, chunk, status, workspace)
    return _head_logprobs(h, W, tokens, chunk, status, workspace, False)[0]


def head_logprobs_bwd(h, W, tokens, row_stats, entropy, grad_logp=None, grad_entropy=None,
                      grad_lse=None, chunk: int = 4096, want_dh: bool = True,
                      want_dW: bool = True, dW_dtype=torch.float32,
                      dw_group_tokens: int = 16384, workspace=None, stream=None):
    """(dh [N, d] in h's dtype, dW [V, d] in ``dW_dtype``, float32 or h's) of ``head_logprobs``
    for upstream gradients [N] of logp, entropy and lse (None: 0); None for the one that is not
    wanted.  ``row_stats`` [N, 2] and ``entropy`` [N] come from the forward; ``workspace`` and
    ``dw_group_tokens`` as in ``fwd_bwd``."""
    dev = h.device
    kd._on_device(dev, h=h)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return head_logprobs_bwd(h, W, tokens, row_stats, entropy, grad_logp, grad_entropy,
                                     grad_lse, chunk, want_dh, want_dW, dW_dtype,
                                     dw_group_tokens, workspace)
    dt, N, d, V, bits = _head(h, W, tokens, row_stats=row_stats, entropy=entropy)
    _float_rows("row_stats", row_stats, (N, 2))
    _float_rows("entropy", entropy, (N,))
    g = [_upstream(n, x, N, dev) for n, x in (("grad_logp", grad_logp),
                                              ("grad_entropy", grad_entropy),
                                              ("grad_lse", grad_lse))]
    if dW_dtype not in (_F32, W.dtype):
        raise TypeError(f"dW_dtype must be float32 or {W.dtype}")
    wt = _CODES[dW_dtype]
    workspace = _scratch(workspace, head_logprobs_bwd_workspace_bytes(
        N, d, V, chunk, dt, wt, dw_group_tokens) if workspace is None else 0, dev)
    dh = torch.empty((N, d), dtype=h.dtype, device=dev) if want_dh else None
    dW = torch.empty((V, d), dtype=dW_dtype, device=dev) if want_dW else None
    kd._check(kd._lib().kd_head_logprobs_bwd(
        h.data_ptr(), W.data_ptr(), dt, tokens.data_ptr(), bits, N, d, V, chunk,
        row_stats.data_ptr(), entropy.data_ptr(), kd._ptr(g[0]), kd._ptr(g[1]), kd._ptr(g[2]),
        kd._ptr(dh), kd._ptr(dW), wt, workspace.data_ptr(), workspace.numel(),
        _raw_stream(dev)))
    return dh, dW


class _HeadLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, tokens, chunk, status, workspace):
        ctx.set_materialize_grads(False)
        outs, st = _head_logprobs(h, W, tokens, chunk, status, workspace, True)
        ctx.save_for_backward(h, W, tokens, outs[1])
        ctx.row_stats = st
        ctx.chunk = chunk
        return outs

    @staticmethod
    def backward(ctx, *grads):
        return (_head_backward_once if torch.is_grad_enabled() else _head_backward)(ctx, *grads)


def _head_backward(ctx, g_logp, g_entropy, g_lse):
    h, W, tokens, entropy = ctx.saved_tensors
    dev = h.device
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _head_backward(ctx, g_logp, g_entropy, g_lse)
    N, d = h.shape
    V = W.shape[0]
    code = _CODES[h.dtype]
    g = _f32(g_logp), _f32(g_entropy), _f32(g_lse)
    dh = torch.empty((N, d), dtype=h.dtype, device=dev) if ctx.needs_input_grad[0] else None
    dW = torch.empty((V, d), dtype=W.dtype, device=dev) if ctx.needs_input_grad[1] else None
    need = head_logprobs_bwd_workspace_bytes(N, d, V, ctx.chunk, code, code)
    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    kd._check(kd._lib().kd_head_logprobs_bwd(
        h.data_ptr(), W.data_ptr(), code, tokens.data_ptr(),
        64 if tokens.dtype is torch.int64 else 32, N, d, V, ctx.chunk, ctx.row_stats.data_ptr(),
        entropy.data_ptr(), kd._ptr(g[0]), kd._ptr(g[1]), kd._ptr(g[2]), kd._ptr(dh),
        kd._ptr(dW), code, workspace.data_ptr(), need, _raw_stream(dev)))
    return dh, dW, None, None, None, None


_head_backward_once = torch.autograd.function.once_differentiable(_head_backward)


# ---- gradient norm and clipping -------------------------------------------------------------
# what is asked of each of many tensors: unbound, as map calls these faster than a loop would
_device_of, _contiguous = torch.Tensor.get_device, torch.Tensor.is_contiguous
_numel, _address, _dtype_of = torch.Tensor.numel, torch.Tensor.data_ptr, operator.attrgetter("dtype")


def _clip(grads, max_norm, out, workspace, stream):
    if not grads:
        raise ValueError("no tensors")
    dev = grads[0].device
    kd._on_device(dev, grads=grads[0])
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _clip(grads, max_norm, out, workspace, None)
    n = len(grads)
    if out is not None and len(out) != n:
        raise ValueError(f"{len(out)} outputs for {n} gradients")
    for name, ts in (("grads", grads), ("out", out or ())):
        if (list(map(_device_of, ts)).count(dev.index) != len(ts)
                or list(map(_contiguous, ts)).count(True) != len(ts)):
            for i, t in enumerate(ts):
                kd._on_device(dev, **{f"{name}[{i}]": t})
                if not t.is_contiguous():
                    raise ValueError(f"{name}[{i}] must be contiguous")
    try:
        types = [_CODES[d] for d in map(_dtype_of, grads)]
    except KeyError as e:
        raise TypeError(f"gradients must be bfloat16 or float32, not {e.args[0]}") from None
    sizes = list(map(_numel, grads))
    if out is not None and (sizes != list(map(_numel, out))
                            or types != list(map(_CODES.get, map(_dtype_of, out)))):
        raise ValueError("out must have the shapes and dtypes of grads")
    held = [array.array("q", sizes), array.array("i", types),
            array.array("Q", map(_address, grads)), array.array("Q", map(_address, out or ()))]
    numel, types, gp, op = (a.buffer_info()[0] for a in held)
    op = op if out is not None else None
    if workspace is None:
        need = ctypes.c_size_t(0)
        kd._check(kd._lib().kd_clip_grads_workspace_bytes(numel, n, ctypes.byref(need)))
        workspace = torch.empty(need.value, dtype=torch.uint8, device=dev)
    else:
        kd._check_workspace(workspace, dev)
    norm = torch.empty(1, dtype=_F32, device=dev)
    kd._check(kd._lib().kd_clip_grads(gp, op, numel, types, n, max_norm, norm.data_ptr(),
                                      workspace.data_ptr(), workspace.numel(),
                                      _raw_stream(dev)))
    return norm


def grad_norm(grads, workspace=None, stream=None):
    """The global norm [1] (float32) of a list of contiguous bfloat16 or float32 CUDA tensors,
    mixed as they come: sqrt of the sum of all squares, summed in float64."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    return _clip(grads, float("inf"), None, workspace, stream)


@torch.no_grad()
def clip_grads(grads, max_norm: float, out=None, workspace=None, stream=None):
    """Clips gradients to a global norm (kd_clip_grads): returns the norm [1] (float32) before
    clipping; where it exceeds ``max_norm`` (and is finite) every tensor is scaled by
    max_norm / norm, in place or into ``out``, tensors of the same shapes and types (which
    get the gradients as they are otherwise).  ``grads`` as in ``grad_norm``; a tensor may
    not appear twice."""
    grads = [grads] if isinstance(grads, torch.Tensor) else list(grads)
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
    norm = _clip(grads, float(max_norm), out, workspace, stream)
    # written behind autograd's back: a backward that saved one of these must notice
    torch.autograd.graph.increment_version(
        [t for t in (grads if out is None else out) if not t.is_inference()])
    return norm
