"""lazy_score_matrix_gb300: streamed pairwise score consumers on GB300 (sm_103a).

A pairwise score S[i,j] = f(x_i, y_j) is evaluated tile by tile in libtp's CUDA kernels, consumed in
the same pass and never stored; first derivatives replay the pairs (torchpairwise guide "Using
Torchpairwise in Models"). Score rows that a model has stored (its logits) have consumers of their own:
token_logprobs and topk_distillation. The C ABI is include/tp.h and include/tp_logits.h; this package is its
Python binding.
"""
from . import masks
from .lazy import LazyScores, TopK, lazy, svgd_direction
from .logits import TokenLogprobs, token_logprobs, topk_distillation, topk_distillation_grad
from .losses import mmd_statistics, sinkhorn_divergence
from .ops import Score

__all__ = ["LazyScores", "TopK", "lazy", "svgd_direction", "mmd_statistics", "sinkhorn_divergence", "Score", "masks",
           "TokenLogprobs", "token_logprobs", "topk_distillation", "topk_distillation_grad"]
