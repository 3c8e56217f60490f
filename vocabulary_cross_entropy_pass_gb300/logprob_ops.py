"""Log-probabilities and distillation on torch tensors, through the C ABI (include/ce.h; the
marshalling is csrc/ce_torch.cpp), and their torch.autograd forms.

  ce_logprobs_fwd, ce_logprobs_bwd    given tokens' log-probabilities, the entropy, the likeliest
                                      tokens; the gradient through the first two
  ce_distill_fwd_bwd                  divergence from a teacher's top logits, loss and gradient
  ce_distill_fwd, ce_distill_bwd      the same in two steps
  token_logprobs, distillation_loss   the same under autograd

Arguments and streams as in vocab_ops.py.  Rows are those of (N, V) or (dim0, dim1, V) logits;
a list of tokens has the rows' shape (one token each) or one dimension more.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib, vocab_ops
from .vocab_ops import _CODE, _load


# ---------------------------------------------------------------- log-probabilities
def ce_logprobs_workspace_bytes(N: int, V: int, dtype: torch.dtype, top_k: int = 0) -> int:
    return int(_lib.load().ce_logprobs_workspace_bytes(N, V, _CODE[dtype], top_k))


def ce_logprobs_fwd(logits: torch.Tensor, tokens: torch.Tensor | None = None, top_k: int = 0,
                    entropy: bool = False, stats: bool = False, ignore_idx: int = -100,
                    workspace: torch.Tensor | None = None, stream=None):
    """``(logprobs, entropy, top_tokens, top_logprobs, stats)``, None for what was not asked:
    the log-probabilities of the given ``tokens`` (their shape, float32; at most 1024 a row), the
    rows' entropies, the ``top_k`` (at most 256) likeliest tokens in falling order (equal logits: the
    lower token first) with their log-probabilities (the rows' shape and top_k), and what
    :func:`ce_logprobs_bwd` needs, (N, 4).

    ``ignore_idx`` among the tokens gives 0; a row of nothing else is not read (zeros, and
    ignore_idx as its top tokens).  Any other token outside [0, V) gives NaN, and the error word
    that ce_get_error reads from a ``workspace`` handed in.  A row of -inf throughout (a mask that
    allows nothing) gives -inf, entropy 0 and top tokens 0, 1, 2, ..."""
    return (vocab_ops._ext or _load()).logprobs_fwd(logits, tokens, top_k, entropy, stats, ignore_idx, workspace,
                                                    stream)


def ce_logprobs_bwd(logits: torch.Tensor, stats: torch.Tensor, tokens: torch.Tensor | None = None,
                    grad_logprobs: torch.Tensor | None = None, grad_entropy: torch.Tensor | None = None,
                    ignore_idx: int = -100, grad: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of :func:`ce_logprobs_fwd`'s log-probabilities and entropy with respect to the
    logits, from the ``stats`` it gave; the logits must be unchanged since.  ``grad`` may be the
    logits themselves."""
    return (vocab_ops._ext or _load()).logprobs_bwd(logits, stats, tokens, grad_logprobs, grad_entropy, ignore_idx,
                                                    grad, stream)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top_k, entropy, ignore_idx):
        lp, ent, top, top_lp, stats = ce_logprobs_fwd(logits, tokens, top_k=top_k, entropy=entropy, stats=True,
                                                      ignore_idx=ignore_idx)
        ctx.save_for_backward(logits, stats, tokens)
        ctx.ignore_idx = ignore_idx
        ctx.set_materialize_grads(False)
        if top is not None:
            ctx.mark_non_differentiable(top, top_lp)
        return lp, ent, top, top_lp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_lp, grad_ent, *_):
        logits, stats, tokens = ctx.saved_tensors
        if grad_lp is not None and grad_lp.dim() == logits.dim() and grad_lp.shape[-1] == 0:
            grad_lp = None  # lists of no tokens
        if grad_lp is None and grad_ent is None:
            return None, None, None, None, None
        g = ce_logprobs_bwd(logits, stats, tokens, grad_logprobs=_flat(grad_lp), grad_entropy=_flat(grad_ent),
                            ignore_idx=ctx.ignore_idx)
        return g, None, None, None, None


def _flat(g: torch.Tensor | None) -> torch.Tensor | None:
    return g if g is None else g.to(torch.float32).contiguous()


def _rows(logits: torch.Tensor) -> torch.Tensor:
    return logits if logits.stride(-1) == 1 else logits.contiguous()


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None = None, top_k: int = 0, entropy: bool = False,
                   ignore_idx: int = -100):
    """:func:`ce_logprobs_fwd` with autograd: ``(logprobs, entropy, top_tokens, top_logprobs)``.  The
    gradient reaches the logits through the given tokens' log-probabilities and the entropy; the
    top tokens are constants (give them as ``tokens`` to train on them)."""
    return _TokenLogprobs.apply(_rows(logits), tokens, int(top_k), bool(entropy), int(ignore_idx))


# ---------------------------------------------------------------- distillation
def ce_distill_workspace_bytes(N: int, V: int, dtype: torch.dtype) -> int:
    return int(_lib.load().ce_distill_workspace_bytes(N, V, _CODE[dtype]))


def ce_distill_fwd_bwd(logits: torch.Tensor, teacher_tokens: torch.Tensor, teacher_logits: torch.Tensor,
                       temperature: float = 1.0, normalize: bool = True, ignore_idx: int = -100,
                       reduce_loss: bool = False, dloss: torch.Tensor | None = None,
                       grad: torch.Tensor | None = None, loss_out: torch.Tensor | None = None,
                       n_non_ignore_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None):
    """``(loss, grad)`` of the divergence of softmax(logits / temperature) from a teacher known by
    its top logits: ``teacher_tokens`` int64 and ``teacher_logits`` (float32, bfloat16 or float16),
    the rows' shape and K (at most 1024),

      q = softmax(teacher_logits / temperature) over the K, or exp(...) as it is without
          ``normalize`` (log-probabilities; what is not listed takes no part)
      loss = temperature^2 * sum_k q_k (log q_k - log p[teacher_tokens_k])

    per row, or the mean over the rows that count (``reduce_loss``).  A row whose first token is
    ``ignore_idx`` is ignored; a later ignore_idx leaves that entry out.  Any other token outside
    [0, V): loss NaN, zero gradient.  ``dloss``, ``loss_out``, ``n_non_ignore_out``: as for
    ce_fwd_bwd.  ``grad`` (allocated when None) may be the logits themselves."""
    if grad is False:
        raise TypeError("grad must be a tensor or None (ce_distill_fwd has no gradient)")
    return (vocab_ops._ext or _load()).distill_fwd(logits, teacher_tokens, teacher_logits, temperature, normalize,
                                                   ignore_idx, reduce_loss, dloss, grad, False, loss_out,
                                                   n_non_ignore_out, workspace, stream)


def ce_distill_fwd(logits: torch.Tensor, teacher_tokens: torch.Tensor, teacher_logits: torch.Tensor,
                   temperature: float = 1.0, normalize: bool = True, ignore_idx: int = -100,
                   reduce_loss: bool = False, stats: bool = False, loss_out: torch.Tensor | None = None,
                   n_non_ignore_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """``(loss, stats)`` of :func:`ce_distill_fwd_bwd` without the gradient; ``stats`` (None unless
    asked for) float32 (N, 4), for :func:`ce_distill_bwd`."""
    return (vocab_ops._ext or _load()).distill_fwd(logits, teacher_tokens, teacher_logits, temperature, normalize,
                                                   ignore_idx, reduce_loss, None, False, stats, loss_out,
                                                   n_non_ignore_out, workspace, stream)


def ce_distill_bwd(logits: torch.Tensor, teacher_tokens: torch.Tensor, teacher_logits: torch.Tensor,
                   stats: torch.Tensor, temperature: float = 1.0, normalize: bool = True, ignore_idx: int = -100,
                   reduce_loss: bool = False, dloss: torch.Tensor | None = None,
                   n_non_ignore: torch.Tensor | None = None, grad: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The gradient from the ``stats`` of :func:`ce_distill_fwd` (and, with ``reduce_loss``, its
    ``n_non_ignore_out``); the other arguments as they were given there.  ``grad`` may be the logits
    themselves."""
    return (vocab_ops._ext or _load()).distill_bwd(logits, teacher_tokens, teacher_logits, stats, temperature,
                                                   normalize, ignore_idx, reduce_loss, dloss, n_non_ignore, grad,
                                                   stream)


class _Distillation(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, teacher, temperature, normalize, reduce_loss, ignore_idx, inplace_grad):
        n = torch.empty(1, dtype=torch.int64, device=logits.device) if reduce_loss else None
        loss, stats = ce_distill_fwd(logits, tokens, teacher, temperature=temperature, normalize=normalize,
                                     ignore_idx=ignore_idx, reduce_loss=reduce_loss, stats=True, n_non_ignore_out=n)
        ctx.save_for_backward(logits, tokens, teacher, stats, n)
        ctx.cfg = (temperature, normalize, reduce_loss, ignore_idx, inplace_grad)
        return loss.view(()) if reduce_loss else loss.view(logits.shape[:-1])

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        logits, tokens, teacher, stats, n = ctx.saved_tensors
        temperature, normalize, reduce_loss, ignore_idx, inplace_grad = ctx.cfg
        g = ce_distill_bwd(logits, tokens, teacher, stats, temperature=temperature, normalize=normalize,
                           ignore_idx=ignore_idx, reduce_loss=reduce_loss, dloss=_flat(grad_out), n_non_ignore=n,
                           grad=logits if inplace_grad else None)
        if inplace_grad:  # a second pass through this graph, or another reader of the logits in it, is refused
            torch.autograd.graph.increment_version(logits)
        return g, None, None, None, None, None, None, None


def distillation_loss(logits: torch.Tensor, teacher_tokens: torch.Tensor, teacher_logits: torch.Tensor,
                      temperature: float = 1.0, normalize: bool = True, reduce_loss: bool = False,
                      ignore_idx: int = -100, inplace_grad: bool = False) -> torch.Tensor:
    """:func:`ce_distill_fwd` with autograd: the loss of every row (the rows' shape) or the mean.
    The teacher is a constant.  ``inplace_grad``: the gradient overwrites the logits, which the
    caller gives up."""
    return _Distillation.apply(_rows(logits), teacher_tokens, teacher_logits.detach(), float(temperature),
                               bool(normalize), bool(reduce_loss), int(ignore_idx), bool(inplace_grad))
