"""Plain 64-bit forms of the operators around a model's vocabulary and gradients
(embedding, adjusted logits, gradient norm), written from the formulas, with the
error that the kernels' 32-bit arithmetic and single rounding allow."""
import numpy as np
import torch

from model_ref import TINY, UNIT

U32 = 2.0 ** -24


def f32(x):
    """A number as the kernels receive it."""
    return float(np.float32(x))


def embed64(table, tokens, scale):
    """(value, allowed error): the product is rounded to 32 bits, then to the type."""
    t = tokens.reshape(-1).long()
    held = ((t >= 0) & (t < table.shape[0])).unsqueeze(1)
    y = torch.where(held, table.double()[torch.where(held.squeeze(1), t, 0)] * f32(scale), 0.0)
    y = y.reshape(*tokens.shape, table.shape[1])
    return y, y.abs() * (UNIT[table.dtype] + 2 * U32) + TINY[table.dtype]


def embed_backward64(d, tokens, vocab, scale, old=None):
    """(value, allowed error).  A sum of m numbers in 32 bits in any order is off by
    at most (m - 1) 2^-24 times the sum of their magnitudes (to first order, hence m
    here); the product (or the addition to what was there) rounds once to 32 bits
    and once to the type."""
    t = tokens.reshape(-1).long()
    inside = ((t >= 0) & (t < vocab)).nonzero().squeeze(1)
    t, rows = t[inside], d.reshape(-1, d.shape[-1]).double()[inside]
    zero = torch.zeros(vocab, d.shape[-1], dtype=torch.float64, device=d.device)
    total, size = zero.index_add(0, t, rows), zero.index_add(0, t, rows.abs())
    count = torch.zeros(vocab, 1, dtype=torch.float64, device=d.device).index_add_(0, t, torch.ones(t.numel(), 1, dtype=torch.float64, device=d.device))
    y = total * f32(scale)
    error = count * U32 * 1.01 * size * abs(f32(scale))
    if old is not None:
        y = torch.where(count > 0, y + old.double(), old.double())
    error = error + torch.where(count > 0, y.abs() * (UNIT[d.dtype] + 2 * U32) + TINY[d.dtype], 0.0)
    return y, error


def counts_of(history, prompt, vocab):
    """(times generated, whether seen) [rows, vocab] of a history of any integers."""
    rows = history.shape[0]
    c, seen = np.zeros((rows, vocab)), np.zeros((rows, vocab), bool)
    h = history.cpu().numpy().astype(np.int64)
    for r in range(rows):
        given = 0 if prompt is None else int(prompt[r])
        for i, t in enumerate(h[r]):
            if 0 <= t < vocab:
                seen[r, t] = True
                c[r, t] += i >= given
    return torch.from_numpy(c), torch.from_numpy(seen)


def pack(allowed):
    """bool [rows, vocab] -> int32 words, 32 tokens each."""
    rows, vocab = allowed.shape
    a = np.zeros((rows, (vocab + 31) // 32 * 32), np.uint8)
    a[:, :vocab] = allowed.cpu().numpy()
    return torch.from_numpy(np.packbits(a, axis=1, bitorder="little").view(np.int32).copy())


def adjust64(x, history=None, prompt=None, repetition=None, presence=None, frequency=None, bias_tokens=None, bias=None,
             allowed=None):
    """(value, allowed error, factor of the gradient) on the CPU; allowed: bool [rows, vocab].  Each of
    the steps rounds its result to 32 bits, the last one to the type."""
    dtype, (rows, vocab) = x.dtype, x.shape
    y = x.double().cpu()
    error, factor = torch.zeros_like(y), torch.ones_like(y)

    def column(p, default):
        return torch.full((rows, 1), default, dtype=torch.float64) if p is None else p.double().cpu().unsqueeze(1)

    if history is not None:
        c, seen = counts_of(history, prompt, vocab)
        r = column(repetition, 1.0)
        factor = torch.where(seen, torch.where(y > 0, 1.0 / r, r), 1.0)
        y = torch.where(seen, torch.where(y > 0, y / r, y * r), y)
        error = torch.where(seen, y.abs() * U32, 0.0)
        loss = column(frequency, 0.0) * c + column(presence, 0.0)
        y = torch.where(c > 0, y - loss, y)
        error = error + torch.where(c > 0, (loss.abs() + y.abs()) * U32, 0.0)
    if bias is not None:
        ids, b = bias_tokens.cpu().long(), bias.double().cpu()
        for i in range(rows):
            last = {int(t): float(v) for t, v in zip(ids[i], b[i]) if 0 <= int(t) < vocab}
            for t, v in last.items():
                y[i, t] += v
                error[i, t] += abs(float(y[i, t])) * U32
    error = error * 1.01 + y.abs() * UNIT[dtype] * 1.01 + TINY[dtype]
    if allowed is not None:
        y = torch.where(allowed.cpu(), y, float("-inf"))
        factor = torch.where(allowed.cpu(), factor, 0.0)
    return y, torch.where(torch.isfinite(y), error, 0.0), factor


def near(got, want, error):
    """Every finite value within its error, every other one the same."""
    got, want, error = got.detach().double().cpu(), want.cpu(), error.cpu()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), "infinities"
    off = torch.where(fine, (got - want).abs() - error, -1.0)
    worst = int(off.argmax()) if off.numel() else 0
    assert not off.numel() or float(off.max()) <= 0, (worst, float(got.flatten()[worst]), float(want.flatten()[worst]), float(error.flatten()[worst]))
