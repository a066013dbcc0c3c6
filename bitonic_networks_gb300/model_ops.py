"""torch-facing wrappers of libgsort's language-model operators (argument
marshalling only): routing to experts, grouping by expert, moving rows to the
experts and back, and log probabilities of given tokens, with their gradients.

Every call takes CUDA tensors (there is no CPU fallback), runs on the current
stream of their device without synchronising, and returns newly allocated
tensors unless an output is given.  Activations and logits are float32,
bfloat16 or float16; all arithmetic is in 32 bits.  Rows may be strided
(tensor[:, :n] of a wider tensor); the elements of a row are consecutive.
Arguments of a wrong type or shape raise TypeError or ValueError, what the
library refuses raises GsortError.
"""
from __future__ import annotations

import functools
import operator
from typing import NamedTuple

import torch

from . import _lib
from .gsort import GsortError, _workspace

_FLOATS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}


class ExpertGroups(NamedTuple):
    """Pairs (token, slot), numbered token * slots + slot, grouped by expert.

    offsets    [experts + 1] int32  first row of each expert's segment, a multiple of the alignment
    counts     [experts] int32      pairs of each expert
    rows       [capacity] int32     the pair in each row of the layout, -1 where there is none
    positions  [tokens, slots] int32  each pair's row, -1 for a dropped pair
    """
    offsets: torch.Tensor
    counts: torch.Tensor
    rows: torch.Tensor
    positions: torch.Tensor


class TokenLogprobs(NamedTuple):
    """logprobs [rows] and entropy [rows] float32; top_logprobs and top_ids
    [rows, top] (None without alternatives); stats [rows, 2] float32: each
    row's largest logit and its sum of exponentials relative to it."""
    logprobs: torch.Tensor | None
    entropy: torch.Tensor
    top_logprobs: torch.Tensor | None
    top_ids: torch.Tensor | None
    stats: torch.Tensor


def _ptr(t):
    return None if t is None else t.data_ptr()


_entry_points = {}


def _entry(name: str):
    fn = _entry_points.get(name)
    if fn is None:
        fn = _entry_points[name] = getattr(_lib.load(), name)
    return fn


def _call(name: str, device: torch.device, *args):
    """Calls the entry point on the device's current stream.  A single-token
    call costs little more than its launch: the stream's handle is read without
    making a stream object, and the device is switched only where it is another."""
    fn = _entry(name)
    index = device.index
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise GsortError(rc, name)


def _matrix(t: torch.Tensor, name: str):
    """Checks a 2-D float CUDA tensor with consecutive row elements; returns
    (pointer, dtype code, rows, width, row stride)."""
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a CUDA tensor of two dimensions, got {tuple(t.shape)} on {t.device}")
    rows, width = t.shape
    stride, step = t.stride()
    if step != 1 and width > 1:
        raise ValueError(f"the elements of a row of {name} must be consecutive")
    # the stride of a tensor with one row (or none) means nothing
    return t.data_ptr(), code, rows, width, stride if rows > 1 else width


def _flat(t: torch.Tensor, name: str, dtype, shape, device) -> int:
    """Checks a contiguous tensor of the given dtype and shape on the device; returns its pointer."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}")
    return t.data_ptr()


def _int(value, name: str) -> int:
    """An integer that fits the C int it is passed as."""
    value = operator.index(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} is out of range: {value}")
    return value


def _choice(value, table, name):
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {value!r}")
    return code


# ----------------------------------------------------------------- routing
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
    with fewer candidates has experts -1 with weight 0."""
    ptr, code, tokens, experts, stride = _matrix(logits, "logits")
    dev = logits.device
    bias_ptr = None if bias is None else _flat(bias, "bias", torch.float32, (experts,), dev)
    k, groups = _int(k, "k"), _int(groups, "groups")
    kept = groups if groups_kept is None else _int(groups_kept, "groups_kept")
    if k < 1:
        raise ValueError("k must be at least 1")
    how, by = _choice(score, _SCORES, "score"), _choice(group_score, _GROUP_SCORES, "group_score")
    weights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    chosen = torch.empty((tokens, k), dtype=torch.int32, device=dev)
    _call("gsort_route_experts", dev, ptr, code, tokens, experts, stride, bias_ptr, how, groups,
          kept, by, k, 1 if renormalise else 0, scale,
          weights.data_ptr(), chosen.data_ptr())
    return weights, chosen


def route_experts_backward(d_weights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
                           score: str = "softmax", renormalise: bool = False,
                           scale: float = 1.0) -> torch.Tensor:
    """Gradient of route_experts' weights by the logits, for the experts it
    chose; [tokens, experts] of the logits' dtype."""
    ptr, code, tokens, number, stride = _matrix(logits, "logits")
    dev = logits.device
    if experts.dim() != 2:
        raise ValueError("experts must have two dimensions")
    shape = (tokens, experts.shape[1])
    experts_ptr = _flat(experts, "experts", torch.int32, shape, dev)
    d_ptr = _flat(d_weights, "d_weights", torch.float32, shape, dev)
    how = _choice(score, _SCORES, "score")
    out = torch.empty((tokens, number), dtype=logits.dtype, device=dev)
    _call("gsort_route_experts_backward", dev, d_ptr, ptr, code, tokens, number, stride, experts_ptr,
          shape[1], how, 1 if renormalise else 0, scale, out.data_ptr())
    return out


# ---------------------------------------------------- grouping and row moves
@functools.lru_cache(maxsize=1024)
def group_capacity(pairs: int, num_experts: int, align: int = 1) -> int:
    """Rows of the grouped layout that any choice of experts fits into."""
    return int(_entry("gsort_group_capacity")(pairs, num_experts, align))


@functools.lru_cache(maxsize=1024)
def group_workspace_bytes(pairs: int, num_experts: int) -> int:
    return int(_entry("gsort_group_workspace_bytes")(pairs, num_experts))


def group_by_expert(experts: torch.Tensor, num_experts: int, *, align: int = 1,
                    workspace: torch.Tensor | None = None) -> ExpertGroups:
    """Stable grouping of the pairs of experts [tokens, slots] int32 by expert,
    each expert's segment starting at a multiple of `align`.  Pairs whose expert
    is not in 0..num_experts-1 are dropped."""
    if not experts.is_cuda:
        raise ValueError("experts must be a CUDA tensor")
    if experts.dim() != 2:
        raise ValueError("experts must have two dimensions")
    dev = experts.device
    ptr = _flat(experts, "experts", torch.int32, experts.shape, dev)
    num_experts, align = _int(num_experts, "num_experts"), _int(align, "align")
    pairs = experts.numel()
    capacity = group_capacity(pairs, num_experts, align)
    nbytes = group_workspace_bytes(pairs, num_experts)
    ws = _workspace(nbytes, dev, workspace) if nbytes else None
    offsets = torch.empty(max(num_experts, 0) + 1, dtype=torch.int32, device=dev)
    counts = torch.empty(max(num_experts, 0), dtype=torch.int32, device=dev)
    rows = torch.empty(capacity, dtype=torch.int32, device=dev)
    positions = torch.empty_like(experts)
    _call("gsort_group_by_expert", dev, ptr, pairs, num_experts, align, offsets.data_ptr(),
          counts.data_ptr(), rows.data_ptr(), capacity, positions.data_ptr(),
          None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size())
    return ExpertGroups(offsets, counts, rows, positions)


def _layout(groups: ExpertGroups, device):
    """(pointer to positions, pointer to rows, tokens, slots, capacity)"""
    positions, rows = groups.positions, groups.rows
    tokens, k = positions.shape
    return (_flat(positions, "groups.positions", torch.int32, positions.shape, device),
            _flat(rows, "groups.rows", torch.int32, (rows.numel(),), device), tokens, k, rows.numel())


def dispatch_rows(x: torch.Tensor, groups: ExpertGroups) -> torch.Tensor:
    """Copies each token's row of x [tokens, width] to its pairs' rows of the
    grouped layout; rows without a pair are zero.  Returns [capacity, width]."""
    ptr, code, given, width, stride = _matrix(x, "x")
    dev = x.device
    positions, rows, tokens, k, capacity = _layout(groups, dev)
    if given != tokens:
        raise ValueError(f"x must have {tokens} rows, got {given}")
    out = torch.empty((capacity, width), dtype=x.dtype, device=dev)
    _call("gsort_dispatch_rows", dev, ptr, code, tokens, width, stride, positions, k, rows, capacity,
          out.data_ptr())
    return out


def combine_rows(y: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor | None = None) -> torch.Tensor:
    """Sums each token's rows of y [capacity, width] in the grouped layout, with
    weights [tokens, slots] float32 (None: ones, dispatch_rows' gradient).
    Dropped pairs add nothing.  Returns [tokens, width]."""
    ptr, code, given, width, stride = _matrix(y, "y")
    dev = y.device
    positions, _, tokens, k, capacity = _layout(groups, dev)
    if given != capacity:
        raise ValueError(f"y must have {capacity} rows, got {given}")
    w = None if weights is None else _flat(weights, "weights", torch.float32, (tokens, k), dev)
    out = torch.empty((tokens, width), dtype=y.dtype, device=dev)
    _call("gsort_combine_rows", dev, ptr, code, capacity, width, stride, w, positions, tokens, k,
          out.data_ptr())
    return out


def combine_rows_backward(d_out: torch.Tensor, y: torch.Tensor, groups: ExpertGroups, weights: torch.Tensor):
    """Gradients of combine_rows by y and by the weights: (d_y [capacity,
    width], zero where a row holds no pair; d_weights [tokens, slots])."""
    ptr, code, given, width, stride = _matrix(d_out, "d_out")
    y_ptr, y_code, y_rows, y_width, y_stride = _matrix(y, "y")
    if y_code != code:
        raise TypeError("d_out and y must have one dtype")
    dev = d_out.device
    positions, rows, tokens, k, capacity = _layout(groups, dev)
    if given != tokens or y_rows != capacity or y_width != width or y.device != dev:
        raise ValueError("d_out must be [tokens, width] and y [capacity, width] on one device")
    w = _flat(weights, "weights", torch.float32, (tokens, k), dev)
    d_y = torch.empty((capacity, width), dtype=y.dtype, device=dev)
    d_weights = torch.empty((tokens, k), dtype=torch.float32, device=dev)
    _call("gsort_combine_rows_backward", dev, ptr, code, tokens, width, stride, y_ptr, capacity, y_stride, w,
          positions, k, rows, d_y.data_ptr(), d_weights.data_ptr())
    return d_y, d_weights


# ------------------------------------------------------- log probabilities
def _targets(targets, rows, device):
    if targets is None:
        return None, 0
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"targets must be int32 or int64, got {targets.dtype}")
    _flat(targets, "targets", targets.dtype, (rows,), device)
    return targets.data_ptr(), targets.element_size()


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor | None = None, *, top: int = 0) -> TokenLogprobs:
    """Log probabilities of targets [rows] under softmax(logits [rows, vocab]),
    each row's entropy, and its `top` (at most 32) most likely tokens, from one
    read of the logits.  Logits of -inf are masked.  A negative target gives 0,
    one beyond the vocabulary NaN; alternatives come best first, ties to the
    lower index, with -inf and -1 where a row has too few unmasked logits."""
    ptr, code, rows, vocab, stride = _matrix(logits, "logits")
    dev = logits.device
    at, size = _targets(targets, rows, dev)
    top = _int(top, "top")
    if top < 0:
        raise ValueError("top must not be negative")
    lp = None if targets is None else torch.empty(rows, dtype=torch.float32, device=dev)
    entropy = torch.empty(rows, dtype=torch.float32, device=dev)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=dev)
    top_lp = torch.empty((rows, top), dtype=torch.float32, device=dev) if top else None
    top_ids = torch.empty((rows, top), dtype=torch.int32, device=dev) if top else None
    _call("gsort_token_logprobs", dev, ptr, code, rows, vocab, stride, at, size, top, _ptr(lp),
          entropy.data_ptr(), stats.data_ptr(), _ptr(top_lp), _ptr(top_ids))
    return TokenLogprobs(lp, entropy, top_lp, top_ids, stats)


def token_logprobs_backward(d_logprobs: torch.Tensor | None, d_entropy: torch.Tensor | None,
                            logits: torch.Tensor, targets: torch.Tensor | None, result: TokenLogprobs, *,
                            out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient by the logits of sum(d_logprobs * logprobs + d_entropy *
    entropy), [rows, vocab] of the logits' dtype; `result` is the forward
    call's.  `out` may be the logits themselves.  Without it the gradient's rows
    lie up to 15 bytes apart where the logits' rows do not follow each other."""
    ptr, code, rows, vocab, stride = _matrix(logits, "logits")
    dev = logits.device
    at, size = _targets(targets, rows, dev)
    if d_logprobs is not None and targets is None:
        raise ValueError("d_logprobs needs targets")
    dl = None if d_logprobs is None else _flat(d_logprobs, "d_logprobs", torch.float32, (rows,), dev)
    dh = None if d_entropy is None else _flat(d_entropy, "d_entropy", torch.float32, (rows,), dev)
    entropy = _flat(result.entropy, "result.entropy", torch.float32, (rows,), dev)
    stats = _flat(result.stats, "result.stats", torch.float32, (rows, 2), dev)
    if out is None:
        # rows as far from a 16-byte boundary as the logits' move in whole vectors
        out_stride = vocab + (stride - vocab) % (16 // logits.element_size())
        out = torch.empty((rows, out_stride), dtype=logits.dtype, device=dev)
        out_ptr = out.data_ptr()
        if out_stride != vocab:
            out = out[:, :vocab]
    else:
        out_ptr, out_code, _, _, out_stride = _matrix(out, "out")
        if out_code != code or out.shape != logits.shape or out.device != dev:
            raise ValueError("out must have the logits' dtype, shape and device")
    _call("gsort_token_logprobs_backward", dev, dl, dh, ptr, code, rows, vocab, stride, at, size, entropy,
          stats, out_ptr, out_stride)
    return out
