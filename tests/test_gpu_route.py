"""Routing to experts and its gradient on the GPU, against 64-bit forms: expert
counts on both sides of every lane width, groups that divide lanes or not,
biases, masked rows and experts, ties, strides and unaligned rows.

Tolerances, fixed beforehand: a score's exponent is rounded once (|x - m| up to
about 30, 2^-24 each: 2e-6) and sums have at most 1024 terms in a tree, so
weights are held to 1e-5 of their size; gradients add and multiply a few such
numbers: 3e-5 of the terms that they are made of, and the stored type's unit."""
import numpy as np
import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES, TINY, UNIT, route64, route_weights64, scores64, strided

pytestmark = pytest.mark.gpu


def logits_of(tokens, experts, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(tokens, experts, generator=g) * spread).to(dtype).cuda()


def check(logits, k, least=0.9, **how):
    w, e = gs.route_experts(logits, k, **how)
    w64, e64, gap = route64(logits, k, **how)
    assert w.shape == (logits.shape[0], k) and e.shape == w.shape
    assert w.dtype == torch.float32 and e.dtype == torch.int32
    # differences below a few 32-bit units do not decide a choice that rests on computed scores
    exact = how.get("bias") is None and how.get("group_score", "max") == "max"
    clear = np.ones(len(gap), bool) if exact else (gap > 2e-6)
    assert clear.mean() >= least
    assert np.array_equal(e.cpu().numpy()[clear], e64[clear])
    assert np.allclose(w.cpu().numpy()[clear], w64[clear], rtol=1e-5, atol=1e-30)
    return w, e


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", [1, 2, 7, 8, 31, 32, 33, 60, 64, 65, 128, 160, 256, 300, 512, 1000, 1024])
def test_choice_and_weights(experts, dtype):
    for tokens, k in ((1, 1), (5, min(experts, 8)), (131, min(experts, 32))):
        x = logits_of(tokens, experts, dtype, experts + tokens)
        for score in ("softmax", "sigmoid"):
            for renormalise in (False, True):
                check(x, k, score=score, renormalise=renormalise, scale=2.5 if renormalise else 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts", [8, 16, 24, 32, 33, 60, 64, 100, 128, 160, 200, 256, 300, 512, 1000])
def test_many_tokens(experts, dtype):
    """Tokens that share a warp: 4 to 32 lanes each."""
    bias = torch.randint(-60, 61, (experts,), generator=torch.Generator().manual_seed(1)).cuda() * 0.001
    for tokens, k in ((1025, 1), (1531, 4), (1403, min(experts, 7)), (1100, min(experts, 14))):
        x = logits_of(tokens, experts, dtype, experts + tokens)
        x[5], x[6, 1:], x[-1, ::3] = float("-inf"), float("-inf"), float("nan")
        for how in (dict(score="softmax"), dict(score="sigmoid", renormalise=True), dict(score="sigmoid", bias=bias, renormalise=True)):
            _, e = check(x, k, least=0.85, **how)
            how.pop("bias", None)
            d = torch.randn(tokens, k, generator=torch.Generator().manual_seed(k)).cuda()
            got = gs.route_experts_backward(d, x, e, **how)
            exp, size = gradient64(d.double().cpu().numpy(), x.double().cpu().numpy(), e.cpu().numpy(), how["score"], how.get("renormalise", False), 1.0)
            far = np.abs(got.double().cpu().numpy() - exp)
            assert (far <= 3e-5 * size + UNIT[dtype] * np.abs(exp) + TINY[dtype]).all()


@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (160, 5, 2), (60, 6, 3), (32, 4, 2), (24, 8, 5), (128, 16, 3), (512, 8, 2)])
def test_groups_of_many_tokens(experts, groups, kept):
    k = min(8, experts // groups * kept)
    x = logits_of(1200, experts, torch.float32, groups)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(3)).cuda() * 0.1
    for group_score in ("max", "top2"):
        for b in (None, bias):
            check(x, k, bias=b, score="sigmoid", groups=groups, groups_kept=kept, group_score=group_score, renormalise=True)


def test_ties_of_many_tokens():
    g = torch.Generator().manual_seed(2)
    for experts, k in ((16, 4), (60, 4), (100, 8), (256, 8), (256, 16)):
        x = torch.randint(-2, 3, (1300, experts), generator=g).float().cuda()
        x[0] = 0.0
        want = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        for dtype in DTYPES:
            assert torch.equal(gs.route_experts(x.to(dtype), k)[1].long(), want)
        # differences in the last bits of 32-bit logits decide as well
        y = (x + 3).view(torch.int32) + torch.randint(0, 3, (1300, experts), generator=g, dtype=torch.int32).cuda()
        y = y.view(torch.float32)
        assert torch.equal(gs.route_experts(y, k)[1].long(), torch.sort(y, dim=1, descending=True, stable=True).indices[:, :k])


def test_one_renormalised_expert_has_weight_one_and_no_gradient():
    for tokens in (50, 2000):
        x = logits_of(tokens, 100, torch.float32, tokens)
        for score in ("softmax", "sigmoid"):
            w, e = gs.route_experts(x, 1, score=score, renormalise=True)
            assert (w == 1).all()
            d = torch.randn(tokens, 1, generator=torch.Generator().manual_seed(1)).cuda()
            assert (gs.route_experts_backward(d, x, e, score=score, renormalise=True) == 0).all()


def test_low_sigmoid_scores_are_renormalised():
    """Scores that underflow in 32 bits still have their quotients."""
    x = logits_of(40, 32, torch.float32, 3) - 95.0
    x[20:] -= 300.0
    w, e = check(x, 4, score="sigmoid", renormalise=True)
    assert torch.allclose(w.sum(1), torch.ones(40).cuda(), atol=1e-5)
    d = torch.randn(40, 4, generator=torch.Generator().manual_seed(4)).cuda()
    got = gs.route_experts_backward(d, x, e, score="sigmoid", renormalise=True).double()
    q = w.double()
    want = torch.zeros(40, 32, dtype=torch.float64).cuda().scatter_(1, e.long(), q * (d.double() - (d * q).sum(1, keepdim=True)))
    assert torch.allclose(got, want, atol=1e-5)


@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (160, 5, 2), (96, 32, 9), (64, 2, 1), (512, 16, 3),
                                                 (1024, 4, 3), (60, 6, 3), (8, 8, 3), (1000, 25, 7), (256, 8, 8)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups(experts, groups, kept, group_score):
    k = min(8, experts // groups * kept)
    x = logits_of(203, experts, torch.float32, groups)
    bias = torch.randn(experts, generator=torch.Generator().manual_seed(3)).cuda() * 0.1
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            check(x, k, bias=b, score=score, groups=groups, groups_kept=kept, group_score=group_score, renormalise=True)


def test_ties_go_to_the_lower_index():
    x = torch.zeros(3, 256).cuda()
    x[1, 40], x[1, 200] = -0.0, 1.0
    x[2] = torch.randint(0, 3, (256,), generator=torch.Generator().manual_seed(1)).float()
    for how in ({}, {"bias": torch.zeros(256).cuda()}, {"groups": 8, "groups_kept": 3, "group_score": "top2"}):
        w, e = gs.route_experts(x, 8, score="sigmoid", **how)
        assert e[0].tolist() == list(range(8))
        assert e[1].tolist() == [200, 0, 1, 2, 3, 4, 5, 6] if "groups" not in how else e[1, 0].item() == 200
        if "groups" not in how:
            assert e[2].tolist() == torch.sort(x[2], descending=True, stable=True).indices[:8].tolist()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_rows(dtype, score):
    x = logits_of(64, 60, dtype, 5)
    x[3] = float("-inf")                       # nothing left
    x[4, 5:] = float("-inf")                   # fewer than k
    x[5, ::2] = float("nan")
    x[6] = torch.finfo(dtype).min              # the type's lowest value is a number
    x[7, :50] = torch.finfo(dtype).min
    x[8, 10:] = float("-inf")
    x[9] = float("nan")
    for renormalise in (False, True):
        w, e = gs.route_experts(x, 8, score=score, renormalise=renormalise)
        w64, e64, _ = route64(x, 8, score=score, renormalise=renormalise)
        assert np.array_equal(e.cpu().numpy(), e64)
        ok = np.isfinite(w64)
        assert np.allclose(w.cpu().numpy()[ok], w64[ok], rtol=1e-5, atol=1e-30)
        for t in (3, 9):
            assert (e[t] == -1).all() and (w[t] == 0).all()
        d = torch.randn(64, 8, generator=torch.Generator().manual_seed(2)).cuda()
        dx = gs.route_experts_backward(d, x, e, score=score, renormalise=renormalise)
        assert (dx[3] == 0).all() and (dx[9] == 0).all() and torch.isfinite(dx).all()
        assert (dx[torch.isneginf(x)] == 0).all()


def test_bias_at_infinity_or_nan_masks_an_expert():
    x = logits_of(20, 64, torch.float32, 8)
    bias = torch.zeros(64)
    bias[::2], bias[1] = float("-inf"), float("nan")
    w, e = gs.route_experts(x, 32, bias=bias.cuda(), score="sigmoid")
    assert ((e[:, :31] % 2 == 1) & (e[:, :31] != 1)).all()
    assert (e[:, 31] == -1).all() and (w[:, 31] == 0).all()


def test_groups_whose_experts_are_masked():
    x = logits_of(9, 64, torch.float32, 9)
    x[:, 8:] = float("-inf")                   # one group of eight alive
    x[0, 1:8] = float("-inf")                  # with one expert
    w, e = gs.route_experts(x, 4, score="sigmoid", groups=8, groups_kept=2, group_score="top2")
    assert e[0].tolist() == [0, -1, -1, -1]
    assert ((e[1:] >= 0) & (e[1:] < 8)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (0, 1), (8, 0), (3, 5)])
def test_strided_and_unaligned_rows(dtype, pad, off):
    for experts in (60, 256):
        x = logits_of(37, experts, dtype, pad + off)
        v = strided(x, pad, off)
        for how in (dict(score="softmax"), dict(score="sigmoid", renormalise=True)):
            w, e = gs.route_experts(x, 6, **how)
            wv, ev = gs.route_experts(v, 6, **how)
            assert torch.equal(w, wv) and torch.equal(e, ev)
            d = torch.randn(37, 6, generator=torch.Generator().manual_seed(4)).cuda()
            assert torch.equal(gs.route_experts_backward(d, x, e, **how), gs.route_experts_backward(d, v, e, **how))


def gradient64(d, x, experts, score, renormalise, scale):
    """(gradient, size of its terms)"""
    s = scores64(x, score)
    there = experts >= 0
    at = np.maximum(experts, 0)
    w = np.where(there, np.take_along_axis(s, at, 1), 0.0)
    g = np.where(there, d, 0.0) * scale
    terms = np.abs(g)
    if renormalise:
        total = w.sum(1, keepdims=True)
        q = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
        mean, mean_size = (g * q).sum(1, keepdims=True), (np.abs(g) * q).sum(1, keepdims=True)
        g = np.divide(g - mean, total, out=np.zeros_like(w), where=total > 0)
        terms = np.divide(terms + mean_size, total, out=np.zeros_like(w), where=total > 0)
    dense, size = np.zeros_like(x), np.zeros_like(x)
    if score == "sigmoid":
        slope = w * (1 - w)
        np.add.at(dense, (np.arange(len(x))[:, None], at), np.where(there, g * slope, 0.0))
        np.add.at(size, (np.arange(len(x))[:, None], at), np.where(there, terms * slope, 0.0))
    else:
        np.add.at(dense, (np.arange(len(x))[:, None], at), np.where(there, g * w, 0.0))
        np.add.at(size, (np.arange(len(x))[:, None], at), np.where(there, terms * w, 0.0))
        if not renormalise:
            dense -= s * (g * w).sum(1, keepdims=True)
            size += s * (terms * w).sum(1, keepdims=True)
    return dense, size


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_the_formula(dtype, score, renormalise):
    for tokens, experts, k in ((1, 1, 1), (3, 8, 2), (130, 60, 4), (77, 256, 8), (33, 1000, 32), (5, 33, 33 - 1)):
        x = logits_of(tokens, experts, dtype, experts)
        how = dict(score=score, renormalise=renormalise, scale=1.75)
        _, e = gs.route_experts(x, k, **how)
        e[0, k - 1] = -1                       # an entry without an expert takes no part
        d = torch.randn(tokens, k, generator=torch.Generator().manual_seed(k)).cuda()
        got = gs.route_experts_backward(d, x, e, **how)
        assert got.dtype == dtype and got.is_contiguous()
        exp, size = gradient64(d.double().cpu().numpy(), x.double().cpu().numpy(), e.cpu().numpy(), score, renormalise, 1.75)
        far = np.abs(got.double().cpu().numpy() - exp)
        assert (far <= 3e-5 * size + UNIT[dtype] * np.abs(exp) + TINY[dtype]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_differences(score, renormalise):
    x = logits_of(11, 40, torch.float32, 6)
    how = dict(score=score, renormalise=renormalise, scale=1.5)
    _, e = gs.route_experts(x, 5, **how)
    g = torch.Generator().manual_seed(9)
    d, v = torch.randn(11, 5, generator=g), torch.randn(11, 40, generator=g)
    dx = gs.route_experts_backward(d.cuda(), x, e, **how).double().cpu().numpy()
    x64, v64, e64, step = x.double().cpu().numpy(), v.double().numpy(), e.cpu().numpy(), 1e-5
    up = route_weights64(x64 + step * v64, e64, score, renormalise, 1.5)
    down = route_weights64(x64 - step * v64, e64, score, renormalise, 1.5)
    want = (d.double().numpy() * (up - down)).sum(1) / (2 * step)
    # 40 products of a gradient that is off by 3e-5 of terms of size about 1
    assert np.allclose((dx * v64).sum(1), want, atol=1e-4, rtol=0)


def test_no_tokens():
    x = torch.empty(0, 16).cuda()
    w, e = gs.route_experts(x, 2)
    assert w.shape == (0, 2) and e.shape == (0, 2)
    assert gs.route_experts_backward(w, x, e).shape == (0, 16)


def test_refusals():
    x = torch.zeros(4, 16).cuda()
    for bad in (dict(k=0), dict(k=17), dict(k=2, groups=3), dict(k=2, groups=4, groups_kept=5), dict(k=2, score="tanh"),
                dict(k=2, group_score="mean"), dict(k=2, scale=float("nan")), dict(k=2, groups=4, groups_kept=0), dict(k=2, groups=2 ** 32 + 1)):
        with pytest.raises((ValueError, gs.GsortError)):
            gs.route_experts(x, **bad)
    with pytest.raises(ValueError):
        gs.route_experts(x.cpu(), 2)
    with pytest.raises(ValueError):
        gs.route_experts(x.t(), 2)
    with pytest.raises(TypeError):
        gs.route_experts(x.double(), 2)
    with pytest.raises(TypeError):
        gs.route_experts(x, 2, bias=torch.zeros(16, dtype=torch.float16).cuda())
    with pytest.raises(ValueError):
        gs.route_experts(x, 2, bias=torch.zeros(15).cuda())
    w, e = gs.route_experts(x, 2)
    with pytest.raises(ValueError):
        gs.route_experts_backward(w[:3], x, e)
    with pytest.raises(TypeError):
        gs.route_experts_backward(w, x, e.long())


def test_another_stream():
    x = logits_of(4096, 128, torch.bfloat16, 1)
    w, e = gs.route_experts(x, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w2, e2 = gs.route_experts(x, 8)
    s.synchronize()
    assert torch.equal(w, w2) and torch.equal(e, e2)


def all_scores(x, score):
    """Every expert's score [tokens, experts], as the weights that the operator
    returns where a bias makes it choose 32 experts at a time."""
    s = torch.zeros(x.shape).cuda()
    for first in range(0, x.shape[1], 32):
        some = min(32, x.shape[1] - first)
        bias = torch.zeros(x.shape[1]).cuda()
        bias[first:first + some] = 100.0
        w, e = gs.route_experts(x, some, bias=bias, score=score)
        s.scatter_(1, e.long(), w)
    return s


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts", [16, 60, 100, 256, 1000])
def test_biased_choice_is_by_the_scores_that_are_returned(experts, score):
    """Biases that bring all choice values together: what is left of their
    differences is in the scores' last bits.  The order has to be that of the
    32-bit sums of returned score and bias, bit for bit."""
    k = min(32, experts)
    for tokens in (1, 1100):
        for seed in range(6):
            x = logits_of(1, experts, torch.float32, seed).expand(tokens, -1).contiguous()
            s = all_scores(x, score)[0].cpu().numpy()
            bias = np.float32(2.0 ** -7) - s
            value = s + bias
            assert value.dtype == np.float32 and np.ptp(value) < 1e-6
            want = np.argsort(-value, kind="stable")[:k]
            _, e = gs.route_experts(x, k, bias=torch.from_numpy(bias).cuda(), score=score)
            assert (e.cpu().numpy() == want).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups", [(64, 8), (60, 6), (256, 8)])
def test_biased_groups_are_by_the_scores_that_are_returned(experts, groups, score):
    for tokens in (1, 1100):
        for seed in range(6):
            x = logits_of(1, experts, torch.float32, 30 + seed).expand(tokens, -1).contiguous()
            s = all_scores(x, score)[0].cpu().numpy()
            bias = np.float32(2.0 ** -7) - s
            value = s + bias
            best = -np.sort(-value.reshape(groups, -1), axis=1)
            kept = np.argsort(-(best[:, 0] + best[:, 1]), kind="stable")[:3]
            inside = np.isin(np.arange(experts) // (experts // groups), kept)
            want = np.argsort(-np.where(inside, value, -np.inf), kind="stable")[:8]
            _, e = gs.route_experts(x, 8, bias=torch.from_numpy(bias).cuda(), score=score, groups=groups, groups_kept=3, group_score="top2")
            assert (e.cpu().numpy() == want).all()


@pytest.mark.parametrize("experts", [60, 256, 1000])
def test_float32_gradient_of_far_experts(experts):
    """Softmax gradients of experts that were not chosen are -p times one sum, so
    their quotient with that of an expert at the maximum is e^(x - max).  In
    units of 2^-24: the exponential 2 ulp = 4, its correction 1, and two
    roundings of either gradient 4; x - max is exact here."""
    for tokens in (3, 1100):
        g = torch.Generator().manual_seed(experts)
        x = torch.randint(-80 * 256, 0, (tokens, experts), generator=g).float() / 256 + 16
        x[:, 0] = x[:, 7] = 16.0
        x = x.cuda()
        _, e = gs.route_experts(x, 1)
        assert (e == 0).all()
        dx = gs.route_experts_backward(torch.ones(tokens, 1).cuda(), x, e).double()
        want = torch.exp(x.double() - 16.0)
        far = (dx / dx[:, 7:8] / want - 1).abs()[:, 1:]
        assert far.max() <= 10 * 2.0 ** -24, float(far.max())
