"""The library's language-model operators on torch tensors: routing to experts,
grouping by expert, moving rows to the experts and back, log probabilities
of given tokens, embedding lookup and adjusted logits, with their gradients; and
the norm of many gradients, with clipping.

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


class ClippedGradients(NamedTuple):
    """gradients: the clipped tensors, a list; norm: float32 scalar tensor, their norm before."""
    gradients: list[torch.Tensor]
    norm: torch.Tensor


def _checked(result, name: str):
    """A call's tensors; an int in their place is the status of a refusal."""
    if result.__class__ is int:
        raise GsortError(result, name)
    return result


def _wants_grad(t) -> bool:
    return getattr(t, "requires_grad", False) and torch.is_grad_enabled()


def _refuse_recorded(out, name: str):
    """An output in a graph would keep the node that it has, whose gradient knows nothing of what is written."""
    if _wants_grad(out):
        raise RuntimeError(f"{name} with out takes part in no gradient: call it under torch.no_grad(), or with an out that requires none")


def _written(out):
    """A tensor that a call has written: autograd refuses what it had saved of it."""
    if not out.is_inference():
        increment_version(out)


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
    if out is not None:
        _written(out)
    return grad


# --------------------------------------------------------------- embedding
class _EmbedTokens(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale = table.shape[0], scale
        return embed_tokens(table, tokens, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        tokens, = ctx.saved_tensors
        return embed_tokens_backward(d_out.contiguous(), tokens, ctx.vocab, scale=ctx.scale), None, None


def embed_tokens(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0) -> torch.Tensor:
    """scale * table[tokens] for a table [vocab, width] and int32 or int64 tokens
    of any shape, contiguous; [*tokens.shape, width] of the table's dtype.  A token
    that is not in 0..vocab-1 has a row of zeros and no gradient.  The table's
    gradient is dense."""
    if _wants_grad(table):
        return _EmbedTokens.apply(table, tokens, scale)
    return _checked(_ops.embed_tokens(table, tokens, scale), "gsort_embed_tokens")


def embed_workspace_bytes(tokens: int, vocab: int, width: int, dtype: torch.dtype) -> int:
    """Workspace of embed_tokens_backward for so many tokens and a table of this shape."""
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[dtype]
    return int(_lib.load().gsort_embed_tokens_backward_workspace_bytes(tokens, vocab, width, code))


def embed_tokens_backward(d_out: torch.Tensor, tokens: torch.Tensor, vocab: int, *, scale: float = 1.0,
                          out: torch.Tensor | None = None, accumulate: bool = False,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of embed_tokens by its table of `vocab` rows, for d_out
    [*tokens.shape, width] (contiguous; with tokens of one dimension its rows may
    be strided): each token's rows summed in 32 bits, in an order that tokens and sizes
    give (the same from call to call), times scale.
    Rows of tokens that do not occur are zero.  With accumulate the sums are added
    to `out` [vocab, width], whose other rows stay as they are.  An `out` that
    requires a gradient raises RuntimeError where gradients are recorded."""
    _refuse_recorded(out, "embed_tokens_backward")
    grad = _checked(_ops.embed_tokens_backward(d_out, tokens, vocab, scale, out, accumulate, workspace),
                    "gsort_embed_tokens_backward")
    if out is not None:
        _written(out)
    return grad


# --------------------------------------------------------- adjusted logits
class _AdjustLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, history, prompt, repetition, presence, frequency, bias_tokens, bias, allowed):
        signs = repetition is not None      # what the gradient asks of logits and history
        ctx.save_for_backward(logits if signs else None, history if signs else None, repetition, allowed)
        return adjust_logits(logits, history=history, prompt=prompt, repetition=repetition, presence=presence,
                             frequency=frequency, bias_tokens=bias_tokens, bias=bias, allowed=allowed)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        logits, history, repetition, allowed = ctx.saved_tensors
        d_logits = adjust_logits_backward(d_out.contiguous(), logits, history=history, repetition=repetition, allowed=allowed)
        return d_logits, *[None] * 8


def adjust_logits(logits: torch.Tensor, *, history: torch.Tensor | None = None, prompt: torch.Tensor | None = None,
                  repetition: torch.Tensor | None = None, presence: torch.Tensor | None = None,
                  frequency: torch.Tensor | None = None, bias_tokens: torch.Tensor | None = None,
                  bias: torch.Tensor | None = None, allowed: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Logits [rows, vocab] with penalties, biases and a mask, in this order:

    history [rows, length] int32 or int64 holds the tokens before (entries outside
    the vocabulary are padding), the first prompt [rows] int32 of them given, the
    others generated.  A token of the history has its logit divided by repetition
    [rows] float32 where it is positive and multiplied where not; a token
    generated c > 0 times loses frequency * c + presence ([rows] float32 each).
    bias [rows, entries] float32 is added to the tokens bias_tokens names (int32
    or int64, of the same shape; of several entries for a token the last one holds, entries
    outside the vocabulary are padding).  allowed [rows, ceil(vocab / 32)] int32
    has bit v % 32 of word v // 32 set where token v may follow; the others become
    -inf, which token_logprobs takes as masked.

    For biases before the penalties, make two calls: one with the biases, then one
    in place with the rest.  history, biases and allowed may be expanded from one row.  `out` may be the
    logits themselves, which are then written only where they change; it takes
    part in no gradient (RuntimeError where gradients are recorded and the logits or
    `out` require one).  The result has a gradient by the logits; the adjustments
    have none.  Without `out`, result rows lie up to 15 bytes apart where the
    logits' rows do not follow each other."""
    if any(_wants_grad(t) for t in (repetition, presence, frequency, bias)):
        raise RuntimeError("penalties and biases have no gradient: detach them")
    _refuse_recorded(out, "adjust_logits")
    if _wants_grad(logits):
        if out is not None:
            raise RuntimeError("adjust_logits with out takes part in no gradient: call it under torch.no_grad()")
        return _AdjustLogits.apply(logits, history, prompt, repetition, presence, frequency, bias_tokens, bias, allowed)
    adjusted = _checked(_ops.adjust_logits(logits, history, prompt, repetition, presence, frequency, bias_tokens, bias, allowed, out),
                        "gsort_adjust_logits")
    if out is not None:
        _written(out)
    return adjusted


def adjust_logits_backward(d_out: torch.Tensor, logits: torch.Tensor | None, *, history: torch.Tensor | None = None,
                           repetition: torch.Tensor | None = None, allowed: torch.Tensor | None = None,
                           out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of adjust_logits by its logits, from that by its result.  `out`
    may be d_out itself; one that requires a gradient raises RuntimeError where
    gradients are recorded.  The logits are needed with a repetition only, for
    their signs."""
    _refuse_recorded(out, "adjust_logits_backward")
    grad = _checked(_ops.adjust_logits_backward(d_out, logits, history, repetition, allowed, out),
                    "gsort_adjust_logits_backward")
    if out is not None:
        _written(out)
    return grad


# ----------------------------------------------------------- gradient norm
def gradient_norm(gradients) -> torch.Tensor:
    """Euclidean norm of all elements of a list of tensors (dense, of one device,
    any mix of float32, bfloat16 and float16); a float32 scalar tensor.  It takes
    part in no gradient: tensors that require one raise RuntimeError where
    gradients are recorded."""
    return _checked(_ops.gradient_norm(gradients), "gsort_gradient_norm")


def clip_gradients(gradients, max_norm: float, *, scale: float = 1.0, out=None) -> ClippedGradients:
    """The gradients times scale, and times max_norm / norm where the norm of all
    of them (times scale) is above max_norm; with that norm.  `out` is a list of
    tensors like the gradients, or the gradients themselves (which are then not
    written where nothing changes).  Nothing waits for the device: a NaN among them
    makes every gradient NaN, an infinity the finite gradients 0.  A norm beyond
    float32 is returned as infinity, and the gradients are clipped by what it is."""
    return ClippedGradients(*_checked(_ops.clip_gradients(gradients, max_norm, scale, out), "gsort_clip_gradients"))
