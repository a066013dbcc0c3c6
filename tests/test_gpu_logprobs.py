"""Token log probabilities, entropies, alternatives and their gradient on the
GPU, against 64-bit forms.

Tolerances, fixed beforehand, for logits up to about 20: an exponent
x log2(e) - m log2(e) is off by at most 2^-24 of itself and 2^-25 of x (3e-6 of
the exponential), a sum of V terms has at most V / 512 serial additions (1.5e-5
at V = 131072), so the sum's logarithm is good to 2e-5; the entropy and a
gradient's terms to 5e-5 of their size; stored gradients are rounded once."""
import numpy as np
import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES, TINY, UNIT, logprobs64, strided

pytestmark = pytest.mark.gpu
INF = float("inf")


def logits_of(rows, vocab, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * spread).to(dtype).cuda()


def same(got, want, tol):
    got, want = got.double().cpu().numpy(), want.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    assert (np.abs(got[fine] - want[fine]) <= tol * (1 + np.abs(want[fine]))).all()


def check(x, targets, top):
    r = gs.token_logprobs(x, targets, top=top)
    lp, h, vals, ids = logprobs64(x.double(), targets, top)
    if targets is None:
        assert r.logprobs is None
    else:
        same(r.logprobs, lp, 2e-5)
    same(r.entropy, h, 5e-5)
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids.cpu().numpy())
        same(r.top_logprobs, vals, 2e-5)
    else:
        assert r.top_logprobs is None and r.top_ids is None
    return r


def check_gradient(x, targets, r, seed=0, out=None):
    rows, vocab = x.shape
    g = torch.Generator().manual_seed(seed)
    dl, dh = torch.randn(rows, generator=g).cuda(), torch.randn(rows, generator=g).cuda()
    x64 = x.double()
    for a, b in ((dl, dh), (dl, None), (None, dh)):
        if targets is None and a is not None:
            continue
        got = gs.token_logprobs_backward(a, b, x, targets, r, out=out)
        assert got.dtype == x.dtype and got.shape == x.shape
        part = ~torch.isneginf(x64)
        d = torch.where(part, x64 - x64.amax(1, keepdim=True), 0.0)     # before the logarithm: it is lost beside 1e38
        log_sum = torch.where(part, d.exp(), 0.0).sum(1, keepdim=True).log()
        lp = torch.where(part, d - log_sum, 0.0)
        p = torch.where(part, lp.exp(), 0.0)
        h = -(p * lp).sum(1, keepdim=True)
        zero = torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
        ga = zero if a is None else torch.where(targets >= 0, a, 0.0).double().unsqueeze(1)
        gb = zero if b is None else b.double().unsqueeze(1)
        want = -p * (ga + gb * (lp + h))
        size = p * (ga.abs() + gb.abs() * (lp.abs() + h))
        if targets is not None:
            alive = torch.isfinite(log_sum).double()
            at = targets.long().clamp(min=0).unsqueeze(1)
            want.scatter_add_(1, at, ga * alive)
            size.scatter_add_(1, at, ga.abs() * alive)
        far = (got.double() - want).abs()
        off = ~(far <= 5e-5 * size + UNIT[x.dtype] * want.abs() + TINY[x.dtype])
        assert not bool(off.any()), (off.nonzero()[:4].tolist(), got[off][:4].tolist(), want[off][:4].tolist())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 33, 500, 4096, 4097, 16384, 32001, 100_003, 200_000])
def test_values_and_gradient(dtype, vocab):
    for rows, top in ((1, 32), (3, 5), (9, 0)):
        x = logits_of(rows, vocab, dtype, vocab + rows)
        g = torch.Generator().manual_seed(vocab)
        t = torch.randint(0, vocab, (rows,), generator=g).cuda()
        r = check(x, t, top)
        check_gradient(x, t, r)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_rows(dtype):
    """More rows than the device holds at once: a CTA per row."""
    x = logits_of(700, 3001, dtype, 4)
    t = torch.randint(0, 3001, (700,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    r = check(x, t, 20)
    check_gradient(x, t, r)
    check(logits_of(1300, 5, dtype, 5), None, 3)
    x = logits_of(1300, 3500, dtype, 6)        # a warp to a row of several steps
    x[::7, 100:] = -INF
    r = check(x, None, 7)
    check_gradient(x, None, r)
    check(strided(logits_of(1217, 8001, dtype, 7), 3, 1), None, 8)     # a warp or a CTA, by the type
    check(logits_of(1217, 8001, dtype, 8), None, 9)
    for vocab, top in ((6001, 5), (2400, 20), (4900, 32), (8100, 1)):  # rows that fill the device
        check(logits_of(3700, vocab, dtype, vocab), None, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (8, 0), (5, 3), (3, 7)])
def test_strided_and_unaligned_rows(dtype, pad, off):
    for vocab in (5, 1000, 40_001):
        x = strided(logits_of(6, vocab, dtype, vocab), pad, off)
        t = torch.tensor([0, vocab - 1, 2, 3, 4, 1]).cuda()
        r = check(x, t, 7)
        check_gradient(x, t, r)
        check_gradient(x, t, r, out=torch.empty(6, vocab, dtype=dtype, device="cuda"))
        check_gradient(x, t, r, out=strided(torch.zeros(6, vocab, dtype=dtype, device="cuda"), 2, 1))


def test_gradient_leaves_what_is_beside_its_rows():
    x = logits_of(5, 1001, torch.bfloat16, 3)
    buf = torch.full((5, 1016), 7.0, dtype=torch.bfloat16, device="cuda")
    r = gs.token_logprobs(x, None)
    gs.token_logprobs_backward(None, torch.ones(5).cuda(), x, None, r, out=buf[:, 3:1004])
    assert (buf[:, :3] == 7).all() and (buf[:, 1004:] == 7).all()


def test_gradient_in_place():
    x = logits_of(40, 9001, torch.bfloat16, 6)
    t = torch.randint(0, 9001, (40,)).cuda()
    r = gs.token_logprobs(x, t)
    d = torch.randn(40).cuda()
    want = gs.token_logprobs_backward(d, d, x, t, r)
    got = gs.token_logprobs_backward(d, d, x, t, r, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [37, 5000, 70_001])
def test_masks(dtype, vocab):
    low = torch.finfo(dtype).min
    x = logits_of(16, vocab, dtype, 11)
    x[0] = -INF                                # masked whole
    x[1, 3:] = -INF                            # fewer than the alternatives
    x[2, :vocab // 2] = -INF
    x[3, ::2] = low                            # masked by the type's lowest value
    x[4] = low                                 # nothing but lowest values: uniform
    x[5, 1:] = -INF
    x[6, torch.rand(vocab, generator=torch.Generator().manual_seed(1)).cuda() < 0.99] = -INF
    x[7] = torch.finfo(dtype).max
    x[8, -1] = torch.finfo(dtype).max
    x[9] = 0.0
    x[10] = -0.0
    x[10, 5] = 0.0
    t = torch.zeros(16, dtype=torch.int64).cuda()
    t[2], t[5], t[6] = vocab - 1, 0, 3
    r = check(x, t, 9)
    assert r.top_ids[9].tolist() == list(range(9)) and r.top_ids[10].tolist() == list(range(9))
    assert r.top_ids[0].tolist() == [-1] * 9 and r.entropy[0].item() == 0.0
    check_gradient(x, t, r)
    dx = gs.token_logprobs_backward(torch.ones(16).cuda(), torch.ones(16).cuda(), x, t, r)
    assert (dx[0] == 0).all() and torch.isfinite(dx).all()
    assert (dx[torch.isneginf(x)].float() == 0).all() or t[6] == 3      # a masked target gets its own gradient


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity(dtype):
    x = logits_of(5, 2000, dtype, 12)
    x[1, 700] = float("nan")
    x[2, 3] = INF
    x[3, :] = -INF
    x[3, 9] = float("nan")
    t = torch.tensor([5, 5, 5, 5, 5]).cuda()
    r = gs.token_logprobs(x, t, top=4)
    assert torch.isfinite(r.logprobs[[0, 4]]).all() and torch.isnan(r.logprobs[1:4]).all() and torch.isnan(r.entropy[1:4]).all()
    ids = logprobs64(x.double(), t, 4)[3]
    assert torch.equal(r.top_ids.long(), ids)
    dx = gs.token_logprobs_backward(torch.ones(5).cuda(), None, x, t, r)
    assert torch.isfinite(dx[[0, 4]]).all() and torch.isnan(dx[1:4]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [3000, 60_000])
def test_orders_that_fill_the_candidate_buffer(dtype, vocab):
    """Rising, falling and constant rows, and rows whose largest logits come last."""
    ramp = torch.linspace(-9, 9, vocab).to(dtype)
    late = torch.zeros(vocab)
    late[-3000:] = torch.rand(3000, generator=torch.Generator().manual_seed(2)) + 1
    x = torch.stack([ramp, ramp.flip(0), torch.ones(vocab).to(dtype), late.to(dtype)]).cuda()
    for reps in (1, 120):                      # split rows, and a CTA per row
        y = x.repeat(reps, 1)
        check(y, None, 32)
        check(y, None, 1)


def test_targets():
    x = logits_of(6, 300, torch.float32, 13)
    for dtype in (torch.int32, torch.int64):
        t = torch.tensor([0, -1, -100, 299, 300, 2 ** 31 - 1], dtype=dtype).cuda()
        r = check(x, t, 0)
        assert r.logprobs[1:3].tolist() == [0.0, 0.0] and torch.isnan(r.logprobs[4:]).all()
        dx = gs.token_logprobs_backward(torch.ones(6).cuda(), None, x, t, r)
        assert (dx[1:3] == 0).all() and torch.isnan(dx[4:]).all() and torch.isfinite(dx[0]).all()


def test_gradient_against_differences():
    x = logits_of(4, 50, torch.float32, 14, 1.0)
    x[1, 7:20] = -INF
    t = torch.tensor([3, 2, -1, 49]).cuda()
    g = torch.Generator().manual_seed(15)
    dl, dh, v = torch.randn(4, generator=g).cuda(), torch.randn(4, generator=g).cuda(), torch.randn(4, 50, generator=g).cuda()
    r = gs.token_logprobs(x, t)
    dx = gs.token_logprobs_backward(dl, dh, x, t, r).double()

    def loss(step):
        lp, h, _, _ = logprobs64(x.double() + step * v.double(), t, 0)
        return dl.double() * lp + dh.double() * h

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    # 50 products of entries that are off by 5e-5 of terms of size up to 1
    assert torch.allclose((dx * v.double()).sum(1), want, atol=5e-4, rtol=0)


def test_offsets_beyond_32_bits():
    """Rows that start past 2^32 bytes and 2^31 elements."""
    stride, vocab = 2 ** 31 + 24, 5001
    buf = torch.empty(2 * stride, dtype=torch.bfloat16, device="cuda")
    x = buf.view(2, stride)[:, :vocab]
    x.copy_(logits_of(2, vocab, torch.bfloat16, 16))
    t = torch.tensor([1, vocab - 1]).cuda()
    r = check(x, t, 5)
    check_gradient(x, t, r, out=torch.empty(2, vocab, dtype=torch.bfloat16, device="cuda"))


def test_last_positions_of_a_batch():
    """Rows far apart: the gradient takes no more room than its rows."""
    x = logits_of(6 * 50, 1003, torch.bfloat16, 17).view(6, 50, 1003)[:, -1]
    t = torch.arange(6).cuda()
    r = check(x, t, 3)
    check_gradient(x, t, r)
    dx = gs.token_logprobs_backward(None, torch.ones(6).cuda(), x, t, r)
    assert dx.untyped_storage().nbytes() <= 6 * (1003 + 7) * 2


def test_no_rows():
    x = torch.empty(0, 10).cuda()
    r = gs.token_logprobs(x, torch.empty(0, dtype=torch.int64).cuda(), top=3)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 3)
    assert gs.token_logprobs_backward(r.logprobs, r.entropy, x, torch.empty(0, dtype=torch.int64).cuda(), r).shape == (0, 10)


def test_refusals():
    x, t = torch.zeros(4, 16).cuda(), torch.zeros(4, dtype=torch.int64).cuda()
    with pytest.raises(gs.GsortError):
        gs.token_logprobs(x, t, top=33)
    with pytest.raises(gs.GsortError):
        gs.token_logprobs(torch.empty(4, 0).cuda(), t)
    for bad in (lambda: gs.token_logprobs(x.cpu(), t), lambda: gs.token_logprobs(x, t[:3]), lambda: gs.token_logprobs(x, t, top=-1),
                lambda: gs.token_logprobs(x.t(), None), lambda: gs.token_logprobs(x, t.cpu()), lambda: gs.token_logprobs(x[0], None)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gs.token_logprobs(x, t.float())
    with pytest.raises(TypeError):
        gs.token_logprobs(x.double(), t)
    r = gs.token_logprobs(x, t)
    with pytest.raises(ValueError):
        gs.token_logprobs_backward(r.logprobs, None, x, None, r)
    with pytest.raises(ValueError):
        gs.token_logprobs_backward(r.logprobs, None, x, t, r, out=torch.empty(4, 15).cuda())
    buf = torch.zeros(4 * 17 + 8).cuda()
    with pytest.raises(gs.GsortError):         # overlapping, but not in place
        a = buf[:64].view(4, 16)
        gs.token_logprobs_backward(r.logprobs, None, a, t, r, out=buf[4:68].view(4, 16))


def test_float32_gradient_far_from_the_maximum():
    """A float32 gradient keeps its relative accuracy where probabilities are
    small: against 64 bits from the forward call's own stats and entropy, with
    x - max exact.  In units of 2^-24: the exponential 2 ulp = 4 and its correction
    1, three products and a quotient 4, together 8 (a 2^-21); with the entropy's term
    the factor beside the exponential has 7 more of its terms' size: 16."""
    for vocab, pad in ((37, 0), (4096, 0), (20_001, 1)):
        g = torch.Generator().manual_seed(vocab)
        x = torch.randint(-80 * 256, 1, (5, vocab), generator=g).float() / 256 + 16
        x[:, 0] = 16.0
        x = strided(x.cuda(), pad, 0)
        t = torch.zeros(5, dtype=torch.int64).cuda()
        r = gs.token_logprobs(x, t)
        a = torch.randn(5, generator=g).cuda()
        d, total, h = x.double() - 16.0, r.stats[:, 1:].double(), r.entropy.double().unsqueeze(1)
        p, a64 = d.exp() / total, a.double().unsqueeze(1)
        got = gs.token_logprobs_backward(a, None, x, t, r).double()
        off = ((got + p * a64).abs() / (p * a64.abs()))[:, 1:]
        assert off.max() <= 2.0 ** -21, float(off.max())
        got = gs.token_logprobs_backward(None, a, x, t, r).double()
        size = p * a64.abs() * (d.abs() + (h - total.log()).abs())
        off = (got + p * a64 * (d - total.log() + h)).abs() / size
        assert off.max() <= 2.0 ** -20, float(off.max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [37, 5000, 70_001])
def test_masked_logits_have_no_gradient(dtype, vocab):
    """Exactly zero, but for a masked token that was itself given."""
    x = logits_of(6, vocab, dtype, 21)
    x[0, vocab // 3:] = -INF
    x[1, ::2] = -INF
    x[2] = -INF
    x[3, 1:] = -INF
    t = torch.tensor([0, 0, 0, 0, 2, -1]).cuda()
    r = gs.token_logprobs(x, t)
    ones = torch.ones(6).cuda()
    masked = torch.isneginf(x)
    masked[torch.arange(6), t] = False
    assert masked.sum() > vocab
    for dl, dh in ((ones, ones), (ones, None), (None, ones)):
        dx = gs.token_logprobs_backward(dl, dh, x, t, r)
        assert (dx[masked] == 0).all() and (dx[2] == 0).all() and torch.isfinite(dx).all()
