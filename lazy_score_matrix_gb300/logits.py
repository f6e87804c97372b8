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
The same call gives the same bits; a row by itself and the same row in a batch may differ in the last ones, as its
sums are split over other threads.

The calls are operators of PyTorch's dispatcher: a trace (``torch.jit.trace``, ``make_fx``) holds them, runs them again
on its own inputs and has their gradients. (A trace saved to a file needs ``_lib.logits_binding()`` before it is
loaded: the operators are registered with the binding.) Derivatives are reverse mode, once:
forward-mode tangents and second derivatives are refused.

Under CUDA graph capture, call these as anywhere else: they allocate outputs from PyTorch's allocator and use no
workspace. For a captured backward use leaves of their own (PyTorch ties a leaf to the stream it was first used
on), or ``topk_distillation_grad``, which needs no autograd.
"""
from __future__ import annotations

from collections import namedtuple
from typing import Optional

import torch

from . import _lib

TokenLogprobs = namedtuple("TokenLogprobs", ["logprobs", "entropy", "top_logprobs", "top_ids"])


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, *, temperature: float = 1.0,
                   top: int = 0) -> TokenLogprobs:
    """Log probability of ``tokens`` [...] under softmax(logits / temperature), the entropy of each row, and its
    ``top`` likeliest columns: TokenLogprobs(logprobs [...], entropy [...], top_logprobs [..., top], top_ids
    [..., top]), natural logarithms; logprobs is None without tokens, the top fields are None for top = 0.

    Alternatives descend by logit, ties by ascending column; a row with fewer than ``top`` (at most 128) columns
    above -inf ends in (-inf, -1). A token outside [0, M), such as -1 or -100, leaves its row out: it is not looked at
    and gives zeros, (-inf, -1) and a zero gradient. A row of -inf alone has log probability -inf and entropy 0.

    Differentiable in logprobs and entropy; the alternatives carry no gradient. temperature in [1e-3, 1e3]."""
    return TokenLogprobs(*_lib.logits_binding().token_logprobs(logits, tokens, temperature, top))


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
    not looked at, loss 0, gradient 0. A column listed twice holds both shares. Differentiable in the logits; the
    teacher's list is a constant. Multiply by temperature ** 2 to keep gradients of different temperatures in
    proportion."""
    return _lib.logits_binding().topk_distillation(logits, teacher_ids, teacher_values, temperature, rest)


def topk_distillation_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_values: torch.Tensor,
                           weights: Optional[torch.Tensor] = None, *, temperature: float = 1.0, rest: bool = False,
                           out: Optional[torch.Tensor] = None):
    """(loss [...], gradient [..., M] of sum(weights * loss)) in one call, for row weights [...] known beforehand
    (a mask over the number of tokens, a loss scale; all ones when None). The loss is not weighted. Each row
    comes from memory once for both, so this is the form for training: ``logits.backward(gradient)``.

    out: where the gradient is written; it may be the logits themselves, which are then overwritten, or lie between
    their rows at the same strides (``buffer[:, M:]`` for logits ``buffer[:, :M]``)."""
    return _lib.logits_binding().topk_distillation_grad(logits, teacher_ids, teacher_values, weights, temperature, rest, out)
