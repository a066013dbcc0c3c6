"""Plain 64-bit forms of the language-model operators, for the tests: written
from the formulas, loops and sorts where they are shortest."""
import numpy as np
import torch

UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # rounding of one store
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -24}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def scores64(x, score):
    """x: numpy float64 [T, E]; masked and NaN experts have score 0."""
    part = x > -np.inf
    if score == "sigmoid":
        with np.errstate(over="ignore", invalid="ignore"):
            s = 1.0 / (1.0 + np.exp(-x))
        return np.where(part, s, 0.0)
    y = np.where(part, x, -np.inf)
    m = y.max(1, keepdims=True)
    e = np.where(part, np.exp(np.where(part, y - np.where(np.isfinite(m), m, 0.0), -np.inf)), 0.0)
    total = e.sum(1, keepdims=True)
    return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def route64(logits, k, bias=None, score="softmax", groups=1, groups_kept=None, group_score="max",
            renormalise=False, scale=1.0):
    """(weights, experts, gap): gap [T] is the smallest difference of choice or
    group values that the token's result rests on (0 for exact ties, which
    the index decides)."""
    x = logits.double().cpu().numpy()
    T, E = x.shape
    s = scores64(x, score)
    c = np.where(x > -np.inf, x if bias is None else s + bias.double().cpu().numpy(), -np.inf)
    c = np.where(np.isnan(c), -np.inf, c)
    gap = np.full(T, np.inf)

    def order(v, n):
        at = np.argsort(-v, axis=1, kind="stable")
        best = np.take_along_axis(v, at, 1)[:, :n + 1]
        with np.errstate(invalid="ignore"):
            d = best[:, :-1] - best[:, 1:]
        d = np.where(np.isfinite(d), d, np.inf)
        return at, d.min(1, initial=np.inf)

    kept = groups if groups_kept is None else groups_kept
    if groups > 1 and kept < groups:
        base = c if group_score == "max" or bias is not None else np.where(c > -np.inf, s, -np.inf)
        per = np.sort(base.reshape(T, groups, -1), axis=2)[:, :, ::-1]
        value = per[:, :, 0].copy()
        if group_score == "top2" and per.shape[2] > 1:
            second = per[:, :, 1]
            value = np.where(second > -np.inf, value + np.where(second > -np.inf, second, 0.0), value)
        at, g = order(value, kept)
        gap = np.minimum(gap, g)
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, at[:, :kept], True, 1)
        c = np.where(np.repeat(keep, E // groups, 1), c, -np.inf)
    at, g = order(c, k)
    gap = np.minimum(gap, g)
    at = at[:, :k]
    there = np.take_along_axis(c, at, 1) > -np.inf
    w = np.where(there, np.take_along_axis(s, at, 1), 0.0)
    if renormalise:
        if score == "softmax":       # the same quotient, without the underflow of far experts
            z = np.where(there, np.take_along_axis(x, at, 1), -np.inf)
            m = np.where(there.any(1, keepdims=True), z.max(1, keepdims=True), 0.0)
            w = np.where(there, np.exp(z - m), 0.0)
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return w * scale, np.where(there, at, -1), gap


def route_weights64(x, experts, score, renormalise, scale):
    """Weights of given experts as a function of the logits (numpy float64), for differences."""
    there = experts >= 0
    s = np.where(there, np.take_along_axis(scores64(x, score), np.maximum(experts, 0), 1), 0.0)
    if renormalise:
        total = s.sum(1, keepdims=True)
        s = np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    return s * scale


def group_ref(experts, num_experts, align, capacity):
    e = experts.reshape(-1).cpu().numpy().astype(np.int64)
    offsets, counts = np.zeros(num_experts + 1, np.int64), np.zeros(num_experts, np.int64)
    rows, positions = np.full(capacity, -1, np.int64), np.full(e.size, -1, np.int64)
    inside = (e >= 0) & (e < num_experts)
    counts[:] = np.bincount(e[inside], minlength=num_experts)
    offsets[1:] = np.cumsum(-(-counts // align) * align)
    order = np.argsort(np.where(inside, e, num_experts), kind="stable")[:int(inside.sum())]
    first = np.cumsum(counts) - counts
    place = offsets[e[order]] + np.arange(order.size) - first[e[order]]
    positions[order] = place
    rows[place] = order
    return offsets, counts, rows, positions.reshape(tuple(experts.shape))


def logprobs64(x, targets, top):
    """x: float64 tensor [R, V].  (logprobs, entropy, top_logprobs, top_ids); rows with NaN or +inf give NaN."""
    bad = torch.isnan(x).any(1, keepdim=True) | torch.isposinf(x).any(1, keepdim=True)
    part = ~torch.isneginf(x)
    m = x.amax(1, keepdim=True)
    d = torch.where(part & torch.isfinite(m), x - m, 0.0)
    e = torch.where(part, d.exp(), 0.0)
    total = e.sum(1, keepdim=True)
    lp = torch.where(part, d - total.log(), float("-inf"))
    h = torch.where(total > 0, total.log() - (e * d).sum(1, keepdim=True) / total, 0.0)
    lp, h = torch.where(bad, float("nan"), lp), torch.where(bad, float("nan"), h)
    given = None
    if targets is not None:
        t = targets.long()
        given = lp.gather(1, t.clamp(0, x.shape[1] - 1).unsqueeze(1)).squeeze(1)
        given = torch.where(t >= x.shape[1], float("nan"), torch.where(t < 0, 0.0, given))
    ids = vals = None
    if top:
        y = torch.where(torch.isnan(x), float("-inf"), x).cpu().numpy()
        n = min(top, y.shape[1])
        at = torch.from_numpy(np.argsort(-y, axis=1, kind="stable")[:, :n].copy()).to(x.device)
        there = torch.where(torch.isnan(x), float("-inf"), x).gather(1, at) > float("-inf")
        ids = torch.full((x.shape[0], top), -1, dtype=torch.int64, device=x.device)
        vals = torch.full((x.shape[0], top), float("-inf"), dtype=torch.float64, device=x.device)
        ids[:, :n] = torch.where(there, at, -1)
        vals[:, :n] = torch.where(there, lp.gather(1, at), float("-inf"))
    return given, h.squeeze(1), vals, ids


def strided(t, pad, off=0):
    """The same values in a row-strided view of a wider buffer, `off` elements past an aligned address."""
    rows, width = t.shape
    buf = torch.full((rows * (width + pad) + off + 16,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[off:off + rows * (width + pad)].view(rows, width + pad)[:, :width]
    v.copy_(t)
    return v
