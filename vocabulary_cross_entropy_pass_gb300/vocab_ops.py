"""The operators around the cross-entropy pass on torch tensors, through the C ABI
(include/ce.h; the marshalling is csrc/ce_torch.cpp), and their torch.autograd
forms.

  ce_embed_fwd, ce_embed_bwd             rows of the vocabulary matrix by token; their gradient
  ce_rmsnorm_fwd, ce_rmsnorm_bwd         residual addition + root-mean-square norm, 8-bit output
  ce_logits_process, ce_logits_process_bwd   penalties, biases, grammar mask, temperature
  embedding, rms_norm, process_logits    the same under autograd

The ce_* forms take and return plain tensors and can be captured into a CUDA
graph (pass the outputs and the workspace, or allocate from the graph's pool).
``stream``: a call runs on the current stream or on the one handed in, after what
that stream holds; what the call allocates is of that stream's memory, and the
caller waits for the stream before it reads the outputs on another.
As with every torch.autograd graph, capture a backward only of a forward made
on the capture's own stream, with no older graph of the same leaves alive.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch
from torch.autograd.function import once_differentiable

from . import _lib

_CODE = {torch.float32: _lib.CE_F32, torch.bfloat16: _lib.CE_BF16, torch.float16: _lib.CE_F16}
_QUANT = {None: _lib.CE_QUANT_NONE, torch.float8_e4m3fn: _lib.CE_QUANT_E4M3,
          torch.float8_e5m2: _lib.CE_QUANT_E5M2}
_ext = None


def _load():
    """The module of csrc/ce_torch.cpp; raises if it has not been built."""
    global _ext
    path = os.path.join(_lib.HERE, "_gbce_torch.so")
    _lib.load()  # the library it calls
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("_gbce_torch", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gbce_torch", loader))
    loader.exec_module(module)
    module.set_error(_lib.CEError)
    _ext = module
    return module


# ---------------------------------------------------------------- embedding
def ce_embed_fwd(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0, ignore_idx: int = -100,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """``scale * weight[tokens]`` in the weight's dtype, shape ``(*tokens.shape,
    H)``, computed in float32 and rounded once.  ``ignore_idx`` gives a row of
    zeros, any other token outside [0, V) a row of NaN (and, with a
    ``workspace`` of 256 bytes, the error word that ce_get_error reads)."""
    return (_ext or _load()).embed_fwd(tokens, weight, scale, ignore_idx, out, workspace, stream)


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
    return (_ext or _load()).embed_bwd(grad_out, tokens, num_embeddings, scale, ignore_idx, grad_weight, accumulate,
                                       _CODE.get(grad_dtype, -1), workspace, stream)


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
    """t itself when its rows are contiguous and evenly spaced, else a copy."""
    try:
        (_ext or _load()).row_stride(t)
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
    code = _QUANT.get(quant)
    if code is None:
        raise TypeError(f"quant must be torch.float8_e4m3fn, torch.float8_e5m2 or None, not {quant}")
    return (_ext or _load()).rmsnorm_fwd(x, weight, residual, eps, out, residual_out, code, group_size, scales_out,
                                         stream)


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
    return (_ext or _load()).rmsnorm_bwd(grad_out, h, weight, eps, grad_h, grad_x, grad_weight, workspace, stream)


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
def ce_logits_workspace_bytes(N: int, V: int, dtype: torch.dtype, history_max: int = 0, bias_max: int = 0) -> int:
    """Bytes of workspace that ce_logits_process(_bwd) needs for N rows; 0 without lists and for few columns in all."""
    return int(_lib.load().ce_logits_workspace_bytes(N, V, _CODE[dtype], history_max, bias_max))


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
    ``mask_value`` (default -inf; the cross-entropy pass with smoothing needs a
    finite one, say -3e4).  Tokens outside [0, V) are skipped; a row whose mask allows
    nothing is mask_value throughout."""
    return (_ext or _load()).logits_process(logits, out, workspace, stream, params)


def ce_logits_process_bwd(grad_out: torch.Tensor, logits: torch.Tensor, grad: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None, **params) -> torch.Tensor:
    """Gradient of :func:`ce_logits_process` with respect to the logits, from
    the logits it was given and the same parameters (the biases, the frequency
    and presence penalties, the prompt lengths and mask_value change nothing
    and may be left out).  ``grad`` may be ``grad_out`` itself."""
    return (_ext or _load()).logits_process_bwd(grad_out, logits, grad, workspace, stream, params)


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
    from); the parameters are constants.  Takes no ``out``, ``workspace`` or
    ``stream``: the logits are kept for the backward pass, which runs on the
    forward's stream."""
    for name in ("out", "workspace", "stream"):
        if name in params:
            raise TypeError(f"process_logits takes no {name} (ce_logits_process does)")
    x = logits if logits.stride(-1) == 1 else logits.contiguous()
    return _ProcessLogits.apply(x, params)
