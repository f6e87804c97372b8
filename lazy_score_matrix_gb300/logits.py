"""Consumers of stored score rows: what a model's last layer writes, logits [..., M] with one row per position
and one column per vocabulary entry.

``token_logprobs`` is the row consumer beside ``LazyScores.logsumexp`` and ``LazyScores.topk``: log probability
of a given token, entropy, and the likeliest columns under top-k's tie rule. ``topk_distillation`` is the loss on
such lists: a student's rows against the top columns of a teacher's. Both read each row once, where it lies
(include/tp_logits.h), and their derivatives replay the rows in libtp's backward kernels.

    teacher = token_logprobs(teacher_logits, top=64, temperature=T)
    loss = topk_distillation(student_logits, teacher.top_ids, teacher.top_logprobs, temperature=T, rest=True)

Logits are float32, float16 or bfloat16 CUDA tensors of any leading shape; rows may lie at any stride (a slice of
a padded vocabulary, ``logits[:, :-1]`` of a batch) and are copied only when two strides cannot describe them.
Results are float32, gradients have the logits' type. Columns at -inf are masked: probability 0, never chosen.

Under CUDA graph capture, call these as anywhere else: they allocate outputs from PyTorch's allocator and use no
workspace. For a captured backward use leaves of their own (PyTorch ties a leaf to the stream it was first used
on), or ``topk_distillation_grad``, which needs no autograd.
"""
from __future__ import annotations

from collections import namedtuple
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import ops

TokenLogprobs = namedtuple("TokenLogprobs", ["logprobs", "entropy", "top_logprobs", "top_ids"])


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, temperature: float = 1.0,
                   top: int = 0) -> TokenLogprobs:
    """Log probability of ``tokens`` [...] under softmax(logits / temperature), the entropy of each row, and its
    ``top`` likeliest columns: TokenLogprobs(logprobs [...], entropy [...], top_logprobs [..., top], top_ids
    [..., top]), natural logarithms; logprobs is None without tokens, the top fields are None for top = 0.

    Alternatives descend by logit, ties by ascending column; a row with fewer than ``top`` (at most 128) columns
    above -inf ends in (-inf, -1). A token outside [0, M), such as -1 or -100, leaves its row out: it is not read
    and gives zeros, (-inf, -1) and a zero gradient. A row of -inf alone has log probability -inf and entropy 0.

    Differentiable in logprobs and entropy; the alternatives carry no gradient. temperature in [1e-3, 1e3]."""
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        return TokenLogprobs(*_TokenLogprobsFn.apply(logits, tokens, float(temperature), int(top)))
    return TokenLogprobs(*ops.token_logprobs(logits, tokens, float(temperature), int(top))[:4])


def topk_distillation(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_values: torch.Tensor, *,
                      temperature: float = 1.0, rest: bool = False) -> torch.Tensor:
    """Kullback-Leibler divergence of each student row from its teacher's list: loss [...], natural logarithms.

    teacher_ids, teacher_values [..., K] (K at most 128, any order). rest=False: the values are the teacher's
    scores and q = softmax(values / temperature) over the list. rest=True: they are its log probabilities at this
    temperature (what ``token_logprobs(..., top=K, temperature=...)`` returns), and the columns not listed form one
    more class, q_r = 1 - sum q (0 where that is below 2^-20, which the values' rounding can leave) against the
    student's probability of all of them:

        loss = sum_k q_k (log q_k - log p_k)  [+ q_r (log q_r - log p_r)]      p = softmax(logits / temperature)

    An id outside [0, M) or a value of -inf drops the entry (a shorter list); a row without an entry is left out:
    not read, loss 0, gradient 0. A column listed twice holds both shares. Differentiable in the logits; the
    teacher's list is a constant. Multiply by temperature ** 2 to keep gradients of different temperatures in
    proportion."""
    if isinstance(teacher_values, torch.Tensor) and teacher_values.requires_grad and torch.is_grad_enabled():
        raise ValueError("topk_distillation: the teacher's list is a constant; pass teacher_values.detach()")
    if torch.is_grad_enabled() and isinstance(logits, torch.Tensor) and logits.requires_grad:
        return _TopkDistillationFn.apply(logits, teacher_ids, teacher_values, float(temperature), bool(rest))
    return ops.topk_distillation(logits, teacher_ids, teacher_values, float(temperature), rest)[0]


@torch.no_grad()
def topk_distillation_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_values: torch.Tensor,
                           weights: Optional[torch.Tensor] = None, *, temperature: float = 1.0, rest: bool = False,
                           out: Optional[torch.Tensor] = None):
    """(loss [...], gradient [..., M] of sum(weights * loss)) in one call, for row weights [...] known beforehand
    (a mask over the number of tokens, a loss scale; all ones when None). The loss is not weighted. The row is
    read once for both, so this is the form for training: ``logits.backward(gradient)``.

    out: where the gradient is written; it may be the logits themselves, which are then overwritten."""
    loss, grad = ops.topk_distillation_grad(logits, teacher_ids, teacher_values, weights, float(temperature), rest, out)
    if out is not None:
        torch.autograd.graph.increment_version(out)  # a graph that saved it must not use it any more
    return loss, grad


# The backwards run on autograd's own thread, where a step costs twice what it does on the caller's: what the forward
# has checked is not checked again. Pointers are taken anew: a saved tensor may come back at another address (hooks
# that move saved tensors to the host and back).


def _dense(g):
    return g if g is None or g.is_contiguous() else g.contiguous()


def _once(backward):
    """once_differentiable, whose bookkeeping only a backward under create_graph needs."""
    checked = once_differentiable(backward)

    def run(ctx, *grads):
        return checked(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)

    return run


class _TokenLogprobsFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top):
        kept = ops._rows(logits)[1]
        tokens = ops._side(tokens, torch.int64, "tokens", logits.shape[:-1], logits)
        lp, h, topv, topi, stats = ops.token_logprobs(kept, tokens, temperature, top, want_stats=True)
        ctx.set_materialize_grads(False)
        if top:
            ctx.mark_non_differentiable(topv, topi)
        ctx.save_for_backward(kept, tokens, stats)
        ctx.temperature = temperature
        return lp, h, topv, topi

    @staticmethod
    @_once
    def backward(ctx, g_lp, g_h, _gv, _gi):
        if g_lp is None and g_h is None:
            return None, None, None, None
        logits, tokens, stats = ctx.saved_tensors
        r, logits = ops._rows(logits)
        return ops._logprobs_grad(logits, r, tokens, ctx.temperature, stats, _dense(g_lp), _dense(g_h)), None, None, None


class _TopkDistillationFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, values, temperature, rest):
        r, kept = ops._rows(logits)
        _, ids, values = ops._teacher(kept, r, ids, values)
        loss, stats = ops.topk_distillation(kept, ids, values, temperature, rest, want_stats=True)
        ctx.save_for_backward(kept, ids, values, stats)
        ctx.temperature, ctx.rest = temperature, rest
        return loss

    @staticmethod
    @_once
    def backward(ctx, gl):
        logits, ids, values, stats = ctx.saved_tensors
        r, logits = ops._rows(logits)
        return (ops._distillation_grad(logits, r, ids, values, ctx.temperature, ctx.rest, stats, _dense(gl)),
                None, None, None, None)
