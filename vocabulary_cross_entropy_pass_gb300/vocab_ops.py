"""The operators around the cross-entropy pass: marshalling of torch tensors into
the C ABI (include/ce.h), and their torch.autograd forms.

  ce_embed_fwd, ce_embed_bwd             rows of the vocabulary matrix by token; their gradient
  ce_rmsnorm_fwd, ce_rmsnorm_bwd         residual addition + root-mean-square norm, 8-bit output
  ce_logits_process, ce_logits_process_bwd   penalties, biases, grammar mask, temperature
  embedding, rms_norm, process_logits    the same under autograd

The ce_* forms take and return plain tensors and can be captured into a CUDA
graph (pass the outputs and the workspace, or allocate from the graph's pool).
As with every torch.autograd graph, capture a backward only of a forward made
on the capture's own stream, with no older graph of the same leaves alive.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib

_DTYPE = {torch.float32: _lib.CE_F32, torch.bfloat16: _lib.CE_BF16, torch.float16: _lib.CE_F16}
_QUANT = {None: _lib.CE_QUANT_NONE, torch.float8_e4m3fn: _lib.CE_QUANT_E4M3,
          torch.float8_e5m2: _lib.CE_QUANT_E5M2}


def _raise(st: int, what: str):
    if st != 0:
        raise _lib.CEError(st, what)


# A call of a small decoding step takes longer on the host than on the GPU, so the
# paths below ask torch for as little as they can: the current stream's handle
# without a Stream object, one is_contiguous() before any stride.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(device, stream):
    return _raw_stream(device.index) if stream is None else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(dev, t, name):
    if t is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev} (there is no CPU path)")


def _cuda(t, name):
    """(device, dtype code) of the tensor an operator goes by."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    dt = _DTYPE.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported {name} dtype {t.dtype}")
    return t.device, dt


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _rows(t: torch.Tensor, H: int, name: str):
    """(rows, stride between them) of a (..., H) tensor."""
    if t.dim() == 0 or t.shape[-1] != H:
        raise ValueError(f"{name} must have rows of {H} elements, got {tuple(t.shape)}")
    if H > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous (call .contiguous())")
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    if t.dim() == 1:
        return 1, H
    N = t.numel() // H
    if N == 0:
        return 0, H
    # the leading dimensions step over one common stride
    step, size = None, 1
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = st
        elif st != step * size:
            raise ValueError(f"the rows of {name} must be evenly spaced (call .contiguous())")
        size *= n
    return N, H if step is None else step


def _stride(t: torch.Tensor, H: int, name: str) -> int:
    """Stride between the rows of a (..., H) tensor."""
    return H if t.is_contiguous() and t.shape[-1] == H else _rows(t, H, name)[1]


_UNIT = _lib.i64_array((0, 1))  # strides of a contiguous run taken as one row


def _tokens(tokens: torch.Tensor):
    """(tokens, dim0, dim1, strides) of an int64 tensor of any shape."""
    if tokens.dtype != torch.int64:
        raise TypeError("tokens must be int64")
    if tokens.is_contiguous():
        return tokens, 1, tokens.numel(), _UNIT
    if tokens.dim() == 2:
        return tokens, tokens.shape[0], tokens.shape[1], _lib.i64_array(tokens.stride())
    if tokens.dim() != 1:
        tokens = tokens.reshape(-1)
    return tokens, 1, tokens.shape[0], _lib.i64_array((0, tokens.stride(0)))


# ---------------------------------------------------------------- embedding
def ce_embed_fwd(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, ignore_idx: int = -100,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """``scale * weight[tokens]`` in the weight's dtype, shape ``(*tokens.shape,
    H)``, computed in float32 and rounded once.  ``ignore_idx`` gives a row of
    zeros, any other token outside [0, V) a row of NaN (and, with a
    ``workspace`` of 256 bytes, the error word that ce_get_error reads)."""
    dev, dt = _cuda(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must be (V, H)")
    V, H = weight.shape
    _on(dev, tokens, "tokens")
    flat, d0, d1, ts = _tokens(tokens)
    if out is None:
        out = torch.empty((*tokens.shape, H), dtype=weight.dtype, device=dev)
        os = H
    else:
        _on(dev, out, "out")
        if out.dtype != weight.dtype or tuple(out.shape) != (*tokens.shape, H):
            raise ValueError("out must be (*tokens.shape, H) in the weight's dtype")
        os = _stride(out, H, "out")
    _on(dev, workspace, "workspace")
    rc = _lib.load().ce_embed_fwd(flat.data_ptr(), d0, d1, ts, weight.data_ptr(), dt, V, H,
                                  _stride(weight, H, "weight"), scale, ignore_idx, out.data_ptr(), os,
                                  _ptr(workspace), _bytes(workspace), _stream(dev, stream))
    if rc:
        _raise(rc, "ce_embed_fwd")
    return out


def ce_embed_bwd_workspace_bytes(N: int, H: int, V: int) -> int:
    return int(_lib.load().ce_embed_bwd_workspace_bytes(N, H, V))


def ce_embed_bwd(grad_out: torch.Tensor, tokens: torch.Tensor, num_embeddings: int, scale: float = 1.0,
                 ignore_idx: int = -100, grad_weight: torch.Tensor | None = None, accumulate: bool = False,
                 grad_dtype: torch.dtype = torch.float32, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Gradient of :func:`ce_embed_fwd` with respect to the (num_embeddings, H)
    weight, summed in float32 over equal tokens in a fixed order.
    ``grad_weight`` (allocated in ``grad_dtype`` when None) is float32 or of
    ``grad_out``'s dtype and written whole; with ``accumulate`` (float32 only)
    it is added to, as ce_linear_fwd_bwd adds to the gradient of the same,
    tied matrix.  ``workspace``: ce_embed_bwd_workspace_bytes bytes."""
    dev, dt = _cuda(grad_out, "grad_out")
    _on(dev, tokens, "tokens")
    if grad_out.shape[:-1] != tokens.shape:
        raise ValueError(f"grad_out {tuple(grad_out.shape)} does not match tokens {tuple(tokens.shape)}")
    H = grad_out.shape[-1]
    flat, d0, d1, ts = _tokens(tokens)
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate needs the grad_weight to add to")
        grad_weight = torch.empty((num_embeddings, H), dtype=grad_dtype, device=dev)
        wst = H
    else:
        _on(dev, grad_weight, "grad_weight")
        if tuple(grad_weight.shape) != (num_embeddings, H):
            raise ValueError("grad_weight must be (num_embeddings, H)")
        wst = _stride(grad_weight, H, "grad_weight")
    wdt = _DTYPE.get(grad_weight.dtype)
    if wdt is None or (wdt != _lib.CE_F32 and wdt != dt):
        raise TypeError("grad_weight must be float32 or of grad_out's dtype")
    if accumulate and wdt != _lib.CE_F32:
        raise TypeError("grad_weight accumulates in float32")
    lib = _lib.load()
    if workspace is None:
        need = lib.ce_embed_bwd_workspace_bytes(d0 * d1, H, num_embeddings)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _on(dev, workspace, "workspace")
        need = _bytes(workspace)
    rc = lib.ce_embed_bwd(grad_out.data_ptr(), dt, _stride(grad_out, H, "grad_out"), flat.data_ptr(), d0, d1, ts,
                          num_embeddings, H, scale, ignore_idx, grad_weight.data_ptr(), wdt, wst,
                          1 if accumulate else 0, workspace.data_ptr(), need, _stream(dev, stream))
    if rc:
        _raise(rc, "ce_embed_bwd")
    return grad_weight


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, ignore_idx):
        ctx.save_for_backward(tokens)
        ctx.cfg = (weight.shape[0], weight.dtype, scale, ignore_idx)
        return ce_embed_fwd(tokens, weight, scale=scale, ignore_idx=ignore_idx)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        (tokens,) = ctx.saved_tensors
        V, dtype, scale, ignore_idx = ctx.cfg
        g = ce_embed_bwd(_even(grad_out), tokens, V, scale=scale, ignore_idx=ignore_idx, grad_dtype=dtype)
        return None, g, None, None


def embedding(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              ignore_idx: int = -100) -> torch.Tensor:
    """:func:`ce_embed_fwd` with autograd; ``weight.grad`` is of the weight's
    dtype (summed in float32)."""
    w = weight if weight.stride(-1) == 1 else weight.contiguous()
    return _Embedding.apply(tokens, w, float(scale), int(ignore_idx))


def _even(t: torch.Tensor) -> torch.Tensor:
    """t itself when its rows are evenly spaced and contiguous, else a copy."""
    try:
        _rows(t, t.shape[-1], "")
        return t
    except ValueError:
        return t.contiguous()


# ---------------------------------------------------------------- norm
def ce_rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, out: torch.Tensor | None = None,
                   residual_out: torch.Tensor | None = None, quant: torch.dtype | None = None,
                   group_size: int = 0, scales_out: torch.Tensor | None = None, stream=None):
    """``h = x + residual``, ``y = h * weight / sqrt(mean(h^2) + eps)`` over the
    last dimension.  Returns ``(y, h, scales)``: h is ``x`` itself without a
    residual; scales is None unless ``quant`` (torch.float8_e4m3fn or
    torch.float8_e5m2) asks for y in 8 bits, then float32 ``(rows, ceil(H /
    group_size))`` with ``y = q * scale`` and group_size 32, 64, 128 or 0 (the
    row).  ``weight``: H elements of x's dtype or float32.  ``residual_out`` may
    be x or residual, ``out`` (without quant) too."""
    dev, dt = _cuda(x, "x")
    shape, dtype = x.shape, x.dtype
    if not shape:
        raise ValueError("x must be (..., H)")
    H = shape[-1]
    N = x.numel() // H if H else 0
    _on(dev, weight, "weight")
    wdt = _DTYPE.get(weight.dtype)
    if wdt != dt and wdt != _lib.CE_F32:
        raise TypeError("weight must be of x's dtype or float32")
    if weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous vector of H elements")
    rs = hs = 0
    if residual is not None:
        _on(dev, residual, "residual")
        if residual.shape != shape or residual.dtype != dtype:
            raise ValueError("residual must match x in shape and dtype")
        rs = _stride(residual, H, "residual")
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dtype, device=dev)
    if residual_out is not None:
        _on(dev, residual_out, "residual_out")
        if residual_out.shape != shape or residual_out.dtype != dtype:
            raise ValueError("residual_out must match x in shape and dtype")
        hs = _stride(residual_out, H, "residual_out")
    if quant is None:
        code = 0
        if group_size or scales_out is not None:
            raise ValueError("group_size and scales_out go with quant")
    else:
        code = _QUANT.get(quant)
        if code is None:
            raise TypeError(f"quant must be torch.float8_e4m3fn, torch.float8_e5m2 or None, not {quant}")
        if group_size not in (0, 32, 64, 128):
            raise ValueError("group_size must be 0, 32, 64 or 128")
        G = 1 if group_size == 0 else -(-H // group_size)
        if scales_out is None:
            scales_out = torch.empty((N, G), dtype=torch.float32, device=dev)
        elif scales_out.dtype != torch.float32 or scales_out.numel() != N * G or not scales_out.is_contiguous():
            raise ValueError("scales_out must be contiguous float32 (rows, groups)")
        _on(dev, scales_out, "scales_out")
        dtype = quant
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
        os = H
    else:
        _on(dev, out, "out")
        if out.shape != shape or out.dtype != dtype:
            raise ValueError("out must match x in shape, in x's dtype or quant's")
        os = _stride(out, H, "out")
    rc = _lib.load().ce_rmsnorm_fwd(x.data_ptr(), _ptr(residual), weight.data_ptr(), dt, wdt, N, H,
                                    _stride(x, H, "x"), rs, eps, out.data_ptr(), os, code, group_size,
                                    _ptr(scales_out), _ptr(residual_out), hs, _stream(dev, stream))
    if rc:
        _raise(rc, "ce_rmsnorm_fwd")
    return out, x if residual_out is None else residual_out, scales_out


def ce_rmsnorm_bwd_workspace_bytes(N: int, H: int) -> int:
    return int(_lib.load().ce_rmsnorm_bwd_workspace_bytes(N, H))


def ce_rmsnorm_bwd(grad_out: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                   grad_h: torch.Tensor | None = None, grad_x: torch.Tensor | None = None,
                   grad_weight: torch.Tensor | bool | None = True, workspace: torch.Tensor | None = None,
                   stream=None):
    """Gradients of :func:`ce_rmsnorm_fwd` from the h it returned.  ``grad_h``:
    what reaches h from the residual stream.  Returns ``(grad_x,
    grad_weight)``: grad_x (x's and the residual's alike) in h's dtype, may be
    given as grad_out, h or grad_h; grad_weight float32, None to skip it."""
    dev, dt = _cuda(h, "h")
    shape, dtype = h.shape, h.dtype
    if not shape:
        raise ValueError("h must be (..., H)")
    H = shape[-1]
    N = h.numel() // H if H else 0
    _on(dev, weight, "weight")
    wdt = _DTYPE.get(weight.dtype)
    if wdt != dt and wdt != _lib.CE_F32:
        raise TypeError("weight must be of h's dtype or float32")
    if weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous vector of H elements")
    if grad_x is None:
        grad_x = torch.empty(shape, dtype=dtype, device=dev)
    dhs = 0
    for t, name in ((grad_out, "grad_out"), (grad_h, "grad_h"), (grad_x, "grad_x")):
        if t is not None and (t.shape != shape or t.dtype != dtype or t.device != dev):
            raise ValueError(f"{name} must match h in shape, dtype and device")
    if grad_h is not None:
        dhs = _stride(grad_h, H, "grad_h")
    lib = _lib.load()
    gw, need = None, 0
    if grad_weight is True:
        gw = torch.empty(H, dtype=torch.float32, device=dev)
    elif isinstance(grad_weight, torch.Tensor):
        gw = grad_weight
        _on(dev, gw, "grad_weight")
        if gw.dtype != torch.float32 or gw.shape != (H,) or not gw.is_contiguous():
            raise TypeError("grad_weight must be a contiguous float32 vector of H elements")
    if gw is not None:
        if workspace is None:
            need = lib.ce_rmsnorm_bwd_workspace_bytes(N, H)
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            _on(dev, workspace, "workspace")
            need = _bytes(workspace)
    rc = lib.ce_rmsnorm_bwd(grad_out.data_ptr(), h.data_ptr(), weight.data_ptr(), _ptr(grad_h), dt, wdt, N, H,
                            _stride(grad_out, H, "grad_out"), _stride(h, H, "h"), dhs, eps, grad_x.data_ptr(),
                            _stride(grad_x, H, "grad_x"), _ptr(gw), _ptr(workspace), need, _stream(dev, stream))
    if rc:
        _raise(rc, "ce_rmsnorm_bwd")
    return grad_x, gw


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h, _ = ce_rmsnorm_fwd(x, weight, residual=residual, eps=eps)
        ctx.save_for_backward(h, weight)
        ctx.eps = eps
        ctx.set_materialize_grads(False)
        return (y, h) if residual is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_h=None):
        h, weight = ctx.saved_tensors
        if grad_y is None:
            return grad_h, None, grad_h if ctx.needs_input_grad[2] else None, None
        gx, gw = ce_rmsnorm_bwd(_even(grad_y), h, weight, eps=ctx.eps,
                                grad_h=None if grad_h is None else _even(grad_h),
                                grad_weight=True if ctx.needs_input_grad[1] else None)
        return gx, gw if gw is None else gw.to(weight.dtype), gx if ctx.needs_input_grad[2] else None, None


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6):
    """:func:`ce_rmsnorm_fwd` with autograd: returns y, or ``(y, h)`` with a
    residual (h is the stream's next residual)."""
    return _RMSNorm.apply(_even(x), weight, residual if residual is None else _even(residual), float(eps))


# ---------------------------------------------------------------- logits
_I64x3 = ctypes.c_int64 * 3


def _logits_dims(t: torch.Tensor, name: str):
    """(dim0, dim1, V, strides) of (N, V) or (dim0, dim1, V) logits."""
    s, n = t.stride(), t.shape
    if s and s[-1] != 1 and n[-1] > 1:
        raise ValueError(f"the vocabulary dimension of {name} must be contiguous (call .contiguous())")
    if len(n) == 2:
        return 1, n[0], n[1], _I64x3(n[0] * s[0], s[0], 1)
    if len(n) == 3:
        return n[0], n[1], n[2], _I64x3(s[0], s[1], 1)
    raise ValueError(f"{name} must be (dim0, dim1, V) or (N, V)")


_PER_ROW = (("history_lengths", torch.int64), ("prompt_lengths", torch.int64), ("repetition_penalty", torch.float32),
            ("frequency_penalty", torch.float32), ("presence_penalty", torch.float32), ("temperature", torch.float32))
_LOGITS_PARAMS = {name for name, _ in _PER_ROW} | {"history", "bias_tokens", "bias_values", "mask", "mask_value"}


def _list(t, N, dtype, dev, name):
    """(pointer, stride between rows, entries per row) of an (N, L) list."""
    if t.dtype != dtype or t.device != dev or t.dim() != 2 or t.shape[0] != N:
        raise TypeError(f"{name} must be {dtype} on the logits' device, one row of entries per row of logits")
    L = t.shape[1]
    if t.is_contiguous():
        return t.data_ptr(), L, L
    if L > 1 and t.stride(1) != 1:
        raise ValueError(f"the entries of {name} must be contiguous (call .contiguous())")
    return t.data_ptr(), t.stride(0), L


def _logits_params(N, V, dev, given):
    p = _lib.ce_logits_params()
    if not _LOGITS_PARAMS.issuperset(given):
        raise TypeError(f"unknown parameters {sorted(set(given) - _LOGITS_PARAMS)}")
    get = given.get
    for name, dtype in _PER_ROW:
        t = get(name)
        if t is not None:
            if t.dtype != dtype or t.device != dev or t.numel() != N or not t.is_contiguous():
                raise TypeError(f"{name} must be a contiguous {dtype} CUDA tensor with one value per row")
            setattr(p, name, t.data_ptr())
    history = get("history")
    if history is not None:
        p.history, p.history_stride, p.history_max = _list(history, N, torch.int64, dev, "history")
    elif p.history_lengths or p.prompt_lengths or p.repetition_penalty or p.frequency_penalty or p.presence_penalty:
        raise ValueError("the penalties and lengths need a history")
    tokens, values = get("bias_tokens"), get("bias_values")
    if (tokens is None) != (values is None):
        raise ValueError("bias_tokens and bias_values go together")
    if tokens is not None:
        p.bias_tokens, p.bias_tokens_stride, p.bias_max = _list(tokens, N, torch.int64, dev, "bias_tokens")
        p.bias_values, p.bias_values_stride, n = _list(values, N, torch.float32, dev, "bias_values")
        if n != p.bias_max:
            raise ValueError("bias_tokens and bias_values must have the same shape")
    mask = get("mask")
    if mask is not None:
        words = (V + 31) // 32
        if mask.dtype != torch.int32 or mask.device != dev or mask.shape[-1] != words:
            raise TypeError(f"mask must be int32 on the logits' device with {words} words per row")
        if (mask.dim() == 2 and mask.shape[0] not in (1, N)) or mask.dim() not in (1, 2) or \
                (words > 1 and mask.stride(-1) != 1):
            raise ValueError("mask must be (words,) for all rows or (N, words), its words contiguous")
        p.mask = mask.data_ptr()
        p.mask_stride = mask.stride(0) if mask.dim() == 2 and mask.shape[0] == N and N > 1 else 0
    p.mask_value = get("mask_value", -math.inf)
    return p


def _match(t, like, name):
    if t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must match the logits in shape and dtype, on the same device")


def ce_logits_workspace_bytes(N: int, V: int, dtype: torch.dtype, history_max: int = 0, bias_max: int = 0) -> int:
    """Bytes of workspace that ce_logits_process(_bwd) needs for N rows; 0 without lists and for few columns in all."""
    return int(_lib.load().ce_logits_workspace_bytes(N, V, _DTYPE[dtype], history_max, bias_max))


def _logits_workspace(workspace, p, N, V, dt, dev):
    if workspace is None and (p.history_max or p.bias_max):
        need = _lib.load().ce_logits_workspace_bytes(N, V, dt, p.history_max, p.bias_max)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is None:
        return None, None, 0
    _on(dev, workspace, "workspace")
    return workspace, workspace.data_ptr(), _bytes(workspace)


def ce_logits_process(logits: torch.Tensor, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      stream=None, **params) -> torch.Tensor:
    """The logits a token is taken from: per row of the (N, V) or (dim0, dim1,
    V) ``logits`` (rows flattened to N in the parameters), in float32, rounded
    once,

      z = x / repetition (x > 0) or x * repetition     tokens in the history
      y = (z - frequency * count - presence * [count > 0] + bias) / temperature
      out = y where the mask allows the token, else mask_value

    ``out`` (allocated when None) may be the logits themselves; ``workspace``:
    ce_logits_workspace_bytes bytes (allocated when None).  Parameters,
    each optional: ``history`` int64 (N, L) with ``history_lengths`` int64 (N,)
    tokens in use, the first ``prompt_lengths`` int64 (N,) of them the prompt
    (no count); ``repetition_penalty``, ``frequency_penalty``,
    ``presence_penalty``, ``temperature`` float32 (N,); ``bias_tokens`` int64
    (N, K) and ``bias_values`` float32 (N, K); ``mask`` int32 (N, ceil(V/32)) or
    (ceil(V/32),), bit v % 32 of word v // 32 set where token v is allowed;
    ``mask_value`` (default -inf; the cross-entropy pass needs a finite one,
    say -3e4).  Tokens outside [0, V) are skipped; a row whose mask allows
    nothing is mask_value throughout."""
    dev, dt = _cuda(logits, "logits")
    d0, d1, V, st = _logits_dims(logits, "logits")
    p = _logits_params(d0 * d1, V, dev, params)
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    else:
        _match(out, logits, "out")
    ost = _logits_dims(out, "out")[3]
    workspace, wp, wb = _logits_workspace(workspace, p, d0 * d1, V, dt, dev)
    rc = _lib.load().ce_logits_process(logits.data_ptr(), dt, d0, d1, V, st, ctypes.byref(p), out.data_ptr(), ost, wp, wb, _stream(dev, stream))
    if rc:
        _raise(rc, "ce_logits_process")
    return out


def ce_logits_process_bwd(grad_out: torch.Tensor, logits: torch.Tensor, grad: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None, **params) -> torch.Tensor:
    """Gradient of :func:`ce_logits_process` with respect to the logits, from
    the logits it was given and the same parameters (the biases, the frequency
    and presence penalties, the prompt lengths and mask_value change nothing
    and may be left out).  ``grad`` may be ``grad_out`` itself."""
    dev, dt = _cuda(logits, "logits")
    d0, d1, V, st = _logits_dims(logits, "logits")
    _match(grad_out, logits, "grad_out")
    p = _logits_params(d0 * d1, V, dev, params)
    gst = _logits_dims(grad_out, "grad_out")[3]
    if grad is None:
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    else:
        _match(grad, logits, "grad")
    ost = _logits_dims(grad, "grad")[3]
    workspace, wp, wb = _logits_workspace(workspace, p, d0 * d1, V, dt, dev)
    rc = _lib.load().ce_logits_process_bwd(grad_out.data_ptr(), gst, logits.data_ptr(), dt, d0, d1, V, st,
                                           ctypes.byref(p), grad.data_ptr(), ost, wp, wb, _stream(dev, stream))
    if rc:
        _raise(rc, "ce_logits_process_bwd")
    return grad


_BWD_PARAMS = ("history", "history_lengths", "repetition_penalty", "mask", "temperature")


class _ProcessLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, params):
        keep = [k for k in _BWD_PARAMS if params.get(k) is not None]
        ctx.names = keep
        ctx.save_for_backward(logits, *(params[k] for k in keep))
        return ce_logits_process(logits, **params)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        logits, *rest = ctx.saved_tensors
        g = grad_out if grad_out.stride(-1) == 1 else grad_out.contiguous()
        params = dict(zip(ctx.names, rest))
        if "repetition_penalty" not in params:
            params.pop("history", None)
            params.pop("history_lengths", None)
        return ce_logits_process_bwd(g, logits, **params), None


def process_logits(logits: torch.Tensor, **params) -> torch.Tensor:
    """:func:`ce_logits_process` with autograd: the gradient reaches the logits
    (a policy's log-probabilities under the distribution its tokens were drawn
    from); the parameters are constants."""
    x = logits if logits.stride(-1) == 1 else logits.contiguous()
    return _ProcessLogits.apply(x, params)
