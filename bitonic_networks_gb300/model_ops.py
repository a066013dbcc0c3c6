"""The library's language-model operators on torch tensors: routing to experts,
grouping by expert, moving rows to the experts and back, and log probabilities
of given tokens, with their gradients.

Every call takes CUDA tensors (there is no CPU fallback), runs on the current
stream of their device without synchronising, and returns newly allocated
tensors unless an output is given.  Activations and logits are float32,
bfloat16 or float16; all arithmetic is in 32 bits (include/gsort.h says how
far exponentials are off).  Rows may be strided
(tensor[:, :n] of a wider tensor); the elements of a row are consecutive.
Arguments of a wrong type or shape raise TypeError or ValueError, what the
library refuses raises GsortError.

The forward calls take part in autograd: where gradients are recorded and an
input requires one, their outputs carry it, computed by the backward calls
(which can also be made directly, and record nothing).  There are no second
derivatives, no forward-mode derivatives and no vmap.

The checks, allocations and launches are in the compiled module _ops: a call for
a few tokens takes as long as its host work.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from .gsort import GsortError

_ops = _lib.load_ops()


class ExpertGroups(NamedTuple):
    """Pairs (token, slot), numbered token * slots + slot, grouped by expert.

    offsets    [experts + 1] int32  first row of each expert's segment, a multiple of the alignment
    counts     [experts] int32      pairs of each expert
    rows       [capacity] int32     the pair in each row of the layout, -1 where there is none
    positions  [tokens, slots] int32  each pair's row, -1 for a dropped pair (set to -1 later, it
               drops the pair from the row moves as well: its row counts as without a pair)
    """
    offsets: torch.Tensor
    counts: torch.Tensor
    rows: torch.Tensor
    positions: torch.Tensor


class TokenLogprobs(NamedTuple):
    """logprobs [rows] (None without targets) and entropy [rows] float32;
    top_logprobs and top_ids [rows, top] (None without alternatives); stats
    [rows, 2] float32: each row's largest logit and its sum of exponentials
    relative to it."""
    logprobs: torch.Tensor | None
    entropy: torch.Tensor
    top_logprobs: torch.Tensor | None
    top_ids: torch.Tensor | None
    stats: torch.Tensor


def _checked(result, name: str):
    """A call's tensors; an int in their place is the status of a refusal."""
    if result.__class__ is int:
        raise GsortError(result, name)
    return result


def _wants_grad(t) -> bool:
    return getattr(t, "requires_grad", False) and torch.is_grad_enabled()


# ----------------------------------------------------------------- routing
class _RouteExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, bias, score, groups, groups_kept, group_score, renormalise, scale):
        weights, experts = route_experts(logits, k, bias=bias, score=score, groups=groups, groups_kept=groups_kept,
                                         group_score=group_score, renormalise=renormalise, scale=scale)
        ctx.save_for_backward(logits, experts)
        ctx.how = score, renormalise, scale
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _):
        logits, experts = ctx.saved_tensors
        score, renormalise, scale = ctx.how
        return (route_experts_backward(d_weights.contiguous(), logits, experts, score=score, renormalise=renormalise, scale=scale),
                *[None] * 8)


def route_experts(logits: torch.Tensor, k: int, *, bias: torch.Tensor | None = None,
                  score: str = "softmax", groups: int = 1, groups_kept: int | None = None,
                  group_score: str = "max", renormalise: bool = False, scale: float = 1.0):
    """Chooses k experts for every token from router logits [tokens, experts].

    Scores are a softmax over the experts or a sigmoid each; `bias` [experts]
    float32 is added to the scores for the choice alone; with groups > 1 only
    experts of the groups_kept best groups (by their largest choice value, or
    the sum of their two largest scores) can be chosen.  Experts with a logit
    of -inf or NaN are never chosen.  Returns (weights [tokens, k] float32,
    experts [tokens, k] int32), best first and ties to the lower index; a token
    with fewer candidates has experts -1 with weight 0.  The weights have a
    gradient by the logits; the choice, and so the bias, has none."""
    if _wants_grad(logits):
        return _RouteExperts.apply(logits, k, bias, score, groups, groups_kept, group_score, renormalise, scale)
    return _checked(_ops.route_experts(logits, k, bias, score, groups, groups_kept, group_score, renormalise, scale),
                    "gsort_route_experts")


def route_experts_backward(d_weights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
                           score: str = "softmax", renormalise: bool = False,
                           scale: float = 1.0) -> torch.Tensor:
    """Gradient of route_experts' weights by the logits, for the experts it
    chose; [tokens, experts] of the logits' dtype."""
    return _checked(_ops.route_experts_backward(d_weights, logits, experts, score, renormalise, scale),
                    "gsort_route_experts_backward")


# ---------------------------------------------------- grouping and row moves
def group_capacity(pairs: int, num_experts: int, align: int = 1) -> int:
    """Rows of the grouped layout that any choice of experts fits into."""
    return int(_lib.load().gsort_group_capacity(pairs, num_experts, align))


def group_workspace_bytes(pairs: int, num_experts: int) -> int:
    return int(_lib.load().gsort_group_workspace_bytes(pairs, num_experts))


def group_by_expert(experts: torch.Tensor, num_experts: int, *, align: int = 1,
                    workspace: torch.Tensor | None = None) -> ExpertGroups:
    """Stable grouping of the pairs of experts [tokens, slots] int32 by expert,
    each expert's segment starting at a multiple of `align`.  Pairs whose expert
    is not in 0..num_experts-1 are dropped."""
    return ExpertGroups(*_checked(_ops.group_by_expert(experts, num_experts, align, workspace),
                                  "gsort_group_by_expert"))


class _DispatchRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows, positions):
        ctx.save_for_backward(rows, positions)
        return dispatch_rows(x, ExpertGroups(None, None, rows, positions))

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows):
        return combine_rows(d_rows.contiguous(), ExpertGroups(None, None, *ctx.saved_tensors)), None, None


class _CombineRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, rows, positions):
        ctx.save_for_backward(y, weights, rows, positions)
        return combine_rows(y, ExpertGroups(None, None, rows, positions), weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        y, weights, rows, positions = ctx.saved_tensors
        groups, d_weights, d_out = ExpertGroups(None, None, rows, positions), None, d_out.contiguous()
        if weights is None:
            d_y = dispatch_rows(d_out, groups)
        else:
            d_y, d_weights = combine_rows_backward(d_out, y, groups, weights)
        return d_y, d_weights, None, None


def dispatch_rows(x: torch.Tensor, groups: ExpertGroups) -> torch.Tensor:
    """Copies each token's row of x [tokens, width] to its pairs' rows of the
    grouped layout; rows without a pair are zero.  Returns [capacity, width]."""
    if _wants_grad(x):
        return _DispatchRows.apply(x, groups.rows, groups.positions)
    return _checked(_ops.dispatch_rows(x, groups.positions, groups.rows), "gsort_dispatch_rows")


def combine_rows(y: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor | None = None) -> torch.Tensor:
    """Sums each token's rows of y [capacity, width] in the grouped layout, with
    weights [tokens, slots] float32 (None: ones, dispatch_rows' gradient).
    Dropped pairs add nothing.  Returns [tokens, width]."""
    if _wants_grad(y) or _wants_grad(weights):
        return _CombineRows.apply(y, weights, groups.rows, groups.positions)
    return _checked(_ops.combine_rows(y, groups.positions, groups.rows, weights), "gsort_combine_rows")


def combine_rows_backward(d_out: torch.Tensor, y: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor):
    """Gradients of combine_rows by y and by the weights: (d_y [capacity,
    width], zero where a row holds no pair; d_weights [tokens, slots])."""
    return _checked(_ops.combine_rows_backward(d_out, y, groups.positions, groups.rows, weights),
                    "gsort_combine_rows_backward")


# ------------------------------------------------------- log probabilities
class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, top):
        logprobs, entropy, top_logprobs, top_ids, stats = token_logprobs(logits, targets, top=top)
        # outputs go the same way as inputs: as attributes they would hold their own node for ever
        ctx.save_for_backward(logits, targets, entropy, stats)
        ctx.mark_non_differentiable(stats, *([] if top_ids is None else [top_ids]))
        ctx.set_materialize_grads(False)
        return logprobs, entropy, top_logprobs, top_ids, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, d_logprobs, d_entropy, d_top_logprobs, _ids, _stats):
        if d_top_logprobs is not None:
            raise RuntimeError("top_logprobs have no gradient: give the tokens as targets")
        if d_logprobs is None and d_entropy is None:
            return None, None, None
        logits, targets, entropy, stats = ctx.saved_tensors
        d_logprobs, d_entropy = (None if d is None else d.contiguous() for d in (d_logprobs, d_entropy))
        return token_logprobs_backward(d_logprobs, d_entropy, logits, targets, TokenLogprobs(None, entropy, None, None, stats)), None, None


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, *, top: int = 0) -> TokenLogprobs:
    """Log probabilities of targets [rows] under softmax(logits [rows, vocab]),
    each row's entropy, and its `top` (at most 32) most likely tokens, from one
    read of the logits.  Logits of -inf are masked.  A negative target gives 0,
    one beyond the vocabulary NaN; alternatives come best first, ties to the
    lower index, with -inf and -1 where a row has too few unmasked logits.
    logprobs and entropy have a gradient; going back through top_logprobs raises
    RuntimeError."""
    if _wants_grad(logits):
        return TokenLogprobs(*_TokenLogprobs.apply(logits, targets, top))
    return TokenLogprobs(*_checked(_ops.token_logprobs(logits, targets, top), "gsort_token_logprobs"))


def token_logprobs_backward(d_logprobs: torch.Tensor | None, d_entropy: torch.Tensor | None,
                            logits: torch.Tensor, targets: torch.Tensor | None, result: TokenLogprobs, *,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient by the logits of sum(d_logprobs * logprobs + d_entropy *
    entropy), [rows, vocab] of the logits' dtype; `result` is the forward
    call's.  `out` may be the logits themselves.  Without it the gradient's rows
    lie up to 15 bytes apart where the logits' rows do not follow each other."""
    grad = _checked(_ops.token_logprobs_backward(d_logprobs, d_entropy, logits, targets, result.entropy, result.stats, out),
                    "gsort_token_logprobs_backward")
    if out is not None and not out.is_inference():
        increment_version(out)      # autograd refuses what it had saved of it
    return grad
