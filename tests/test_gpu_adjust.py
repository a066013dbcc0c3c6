"""adjust_logits and its gradient against 64-bit forms: sizes around the pieces of a
row, histories, biases, masks, special values, strides, in place."""
import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES, UNIT, strided
from vocab_ref import U32, adjust64, near, pack

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def inputs(rows, vocab, length, biases, masked, dtype=torch.float32, seed=0, ints=torch.int32):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g) * 2.5).to(dtype)
    how = {}
    if length is not None:
        # some tokens many times, some outside the vocabulary
        h = (torch.rand(rows, length, generator=g) ** 3 * (vocab * 1.1)).long() - 1
        how["history"] = h.to(ints)
        how["prompt"] = torch.randint(-1, length + 2, (rows,), generator=g).to(torch.int32)
        how["repetition"] = 0.8 + torch.rand(rows, generator=g)
        how["presence"], how["frequency"] = torch.randn(rows, generator=g), torch.randn(rows, generator=g)
    if biases is not None:
        how["bias_tokens"] = torch.randint(-2, vocab + 2, (rows, biases), generator=g).to(ints)
        how["bias"] = torch.randn(rows, biases, generator=g) * 4.0
    allowed = (torch.rand(rows, vocab, generator=g) < torch.rand(rows, 1, generator=g)) if masked else None
    return x, how, allowed


def call(x, how, allowed, out=None):
    device = {k: v.cuda() for k, v in how.items()}
    return gs.adjust_logits(x, **device, allowed=None if allowed is None else pack(allowed).cuda(), out=out)


def back(d, x, how, allowed, out=None):
    return gs.adjust_logits_backward(d, x, history=how["history"].cuda() if "history" in how else None,
                                     repetition=how["repetition"].cuda() if "repetition" in how else None,
                                     allowed=None if allowed is None else pack(allowed).cuda(), out=out)


def check(x, how, allowed):
    y, error, factor = adjust64(x, **how, allowed=allowed)
    xs = x.cuda()
    got = call(xs, how, allowed)
    assert got.dtype == x.dtype and got.shape == x.shape
    near(got, y, error)
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).to(x.dtype)
    # 1 / r and the product round to 32 bits, then to the type
    want = d.double() * factor
    near(back(d.cuda(), xs, how, allowed), want, want.abs() * (UNIT[x.dtype] + 3 * U32) + 1e-37)
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 64, 1000, 4095, 4097, 8191, 8192, 8193, 20011])
@pytest.mark.parametrize("length,biases,masked", [(None, None, True), (40, None, False), (None, 7, False), (300, 20, True), (0, 0, True), (1, 1, False)])
def test_sizes(dtype, vocab, length, biases, masked):
    check(*inputs(3, vocab, length, biases, masked, dtype))


@pytest.mark.parametrize("rows,vocab,length", [(1, 40000, 5000), (150, 700, 33), (2, 100003, 20000), (1, 3000, 40000), (2, 30000, 70000),
                                               (3, 5000, 1024), (3, 5000, 4096), (3, 5000, 4097)])
def test_long_histories(rows, vocab, length):
    for ints in (torch.int32, torch.int64):
        check(*inputs(rows, vocab, length, 300, True, torch.bfloat16, ints=ints))


def test_integers_beyond_32_bits_are_no_tokens():
    x = torch.randn(2, 100)
    odd = torch.tensor([[3 + 2 ** 32, -2 ** 32 + 5, 2 ** 63 - 1, 7, -1]] * 2)
    check(x, dict(history=odd, presence=torch.ones(2), repetition=torch.full((2,), 1.5), bias_tokens=odd, bias=torch.randn(2, 5)), None)


def test_many_biases():
    x, how, allowed = inputs(2, 30000, 50, 9000, True)
    check(x, how, allowed)
    spread = torch.arange(0, 30000, 11).repeat(2, 1)           # evenly spaced, all different
    how.update(bias_tokens=spread, bias=torch.randn(spread.shape))
    check(x, how, allowed)


def test_dense_histories():
    """Every token of the vocabulary, some again: the words of the set are full."""
    x, how, allowed = inputs(2, 9000, 20000, 5, True)
    how["history"] = (torch.arange(20000).repeat(2, 1) * 7 % 9000).int()
    check(x, how, allowed)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_dense_histories_in_place(dtype, masked):
    """Full words in one part of the row, single members in another, with the least room for them."""
    x, how, allowed = inputs(2, 40000, 20000, 5, masked, dtype)
    how["history"] = torch.cat([torch.arange(9000), torch.arange(9000, 40000, 37).repeat(13), torch.arange(100)]).repeat(2, 1).int()
    y, error, factor = adjust64(x, **how, allowed=allowed)
    xs = x.cuda()
    near(call(xs, how, allowed, out=xs), y, error)
    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(9)).to(x.dtype)
    ds, want = d.cuda(), d.double() * factor
    near(back(ds, x.cuda(), how, allowed, out=ds), want, want.abs() * (UNIT[dtype] + 3 * U32) + 1e-37)


def test_more_rows_and_vocabulary_than_one_look_takes():
    """Rows of several pieces, each of the largest size: the same row again and again is the row alone."""
    x, how, allowed = inputs(1, 600_000, 3000, 40, True, torch.bfloat16)
    one = call(x.cuda(), how, allowed)
    rows = 310
    many = {k: v.cuda().expand(rows, *v.shape[1:]).contiguous() for k, v in how.items()}
    got = gs.adjust_logits(x.cuda().repeat(rows, 1), **many, allowed=pack(allowed).cuda().expand(rows, -1))
    assert torch.equal(got, one.expand(rows, -1))
    y, error, _ = adjust64(x, **how, allowed=allowed)
    near(one, y, error)


def test_one_token_again_and_again():
    x, how, _ = inputs(2, 50, 3000, None, False)
    how["history"] = torch.full((2, 3000), 7, dtype=torch.int32)
    how["prompt"] = torch.tensor([0, 2999], dtype=torch.int32)
    how["frequency"] = torch.tensor([0.5, 0.5])
    got = check(x, how, None)
    assert torch.equal(got.cpu()[:, :7], x[:, :7])


@pytest.mark.parametrize("given", [("repetition",), ("presence",), ("frequency",), ("prompt",), ()])
def test_single_penalties(given):
    x, how, _ = inputs(4, 500, 60, None, False)
    check(x, {k: v for k, v in how.items() if k == "history" or k in given}, None)


def test_the_last_bias_of_a_token_holds():
    x = torch.zeros(2, 100)
    how = dict(bias_tokens=torch.tensor([[5, 6, 5, -1, 5, 100], [99, 99, 0, 0, 0, 99]]), bias=torch.tensor([[1.0, 2, 3, 4, 5, 6], [1, 2, 3, 4, 5, 6]]))
    got = check(x, how, None).cpu()
    want = torch.zeros(2, 100)
    want[0, 5], want[0, 6], want[1, 99], want[1, 0] = 5, 2, 6, 5
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values(dtype):
    """Masked places may hold anything; elsewhere IEEE arithmetic decides."""
    low = torch.finfo(dtype).min
    x = torch.tensor([[0.0, -0.0, INF, -INF, NAN, low, -low, 1.0] * 8] * 4).to(dtype)
    how = dict(history=torch.arange(0, 64, 2).repeat(4, 1).int(), prompt=torch.tensor([0, 16, 32, 0], dtype=torch.int32),
               repetition=torch.tensor([1.0, 1.5, 1.5, 1.5]), frequency=torch.full((4,), 0.25), presence=torch.full((4,), 0.5),
               bias_tokens=torch.tensor([[1, 3, 9, 11]] * 4), bias=torch.tensor([[INF, 1.0, -INF, 2.0]] * 4))
    allowed = torch.ones(4, 64, dtype=torch.bool)
    allowed[3] = False
    allowed[:, 32:] = False
    big = torch.finfo(dtype).max
    y, error, factor = adjust64(x, **how, allowed=allowed)
    y = torch.where(y.abs() > big * (1 + UNIT[dtype]), y.sign() * INF, y)      # beyond the type
    got = call(x.cuda(), how, allowed)
    near(got, y, torch.where(torch.isfinite(y), error, 0.0))
    assert bool(got[3].isneginf().all()) and bool(got[:, 32:].isneginf().all())
    r = gs.token_logprobs(got, top=3)
    assert float(r.entropy[3]) == 0.0 and r.top_ids[3].tolist() == [-1] * 3
    d = torch.ones_like(got)
    d[:, 40] = NAN
    g = back(d, x.cuda(), how, allowed)
    assert bool((g[3] == 0).all()) and bool((g[:, 32:] == 0).all())
    near(g, factor, factor * (UNIT[dtype] + 3 * U32))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(0, 1), (1, 0), (8, 0), (5, 3), (64, 2)])
def test_strides(dtype, pad, off):
    x, how, allowed = inputs(5, 9001, 200, 30, True, dtype)
    want = call(x.cuda(), how, allowed)
    xs = strided(x.cuda(), pad, off)
    got = call(xs, how, allowed)
    assert torch.equal(got, want) and (got.stride(0) - 9001) * got.element_size() < 16
    for p, o in ((0, 0), (pad, off), (3, 2)):
        out = strided(torch.zeros_like(want), p, o)
        assert call(xs, how, allowed, out=out) is out
        assert torch.equal(out, want)
        if p:
            assert bool(out.as_strided((4, p), (out.stride(0), 1), out.storage_offset() + 9001).isnan().all())
    d = torch.randn_like(want)
    g = back(d, x.cuda(), how, allowed)
    assert torch.equal(back(strided(d, pad, off), strided(x.cuda(), 3, 1), how, allowed, out=strided(d, 7, 1)), g)
    wide = torch.zeros(5, 250, dtype=torch.int32).cuda()       # wider buffers of histories and masks
    wide[:, :200] = how["history"].cuda()
    words = torch.zeros(5, 300, dtype=torch.int32).cuda()
    words[:, 1:283] = pack(allowed).cuda()
    lists = {**{k: v.cuda() for k, v in how.items()}, "history": wide[:, :200]}
    assert torch.equal(gs.adjust_logits(xs, **lists, allowed=words[:, 1:283]), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
@pytest.mark.parametrize("length,biases,masked", [(50, None, False), (None, None, True), (50, 9, True), (None, None, False)])
def test_in_place(dtype, pad, off, length, biases, masked):
    x, how, allowed = inputs(4, 17001, length, biases, masked, dtype)
    if masked:
        allowed[0] = True
        allowed[1] = False
    want = call(x.cuda(), how, allowed)
    xs = strided(x.cuda(), pad, off)
    version = xs._version
    assert call(xs, how, allowed, out=xs) is xs and xs._version > version
    assert torch.equal(xs, want)
    d = torch.randn_like(want)
    g = back(d, x.cuda(), how, allowed)
    ds = strided(d, pad, off)
    assert back(ds, x.cuda(), how, allowed, out=ds) is ds and torch.equal(ds, g)


def test_rows_that_share_their_lists():
    x, how, allowed = inputs(1, 3000, 80, 10, True)
    rows = {k: v for k, v in how.items() if v.dim() == 1}
    many = {k: v.expand(6).contiguous().cuda() for k, v in rows.items()}
    many.update({k: v.cuda().expand(6, -1) for k, v in how.items() if v.dim() == 2})
    words = pack(allowed).cuda().expand(6, -1)
    got = gs.adjust_logits(x.cuda().repeat(6, 1), **many, allowed=words)
    assert torch.equal(got, call(x.cuda(), how, allowed).expand(6, -1))


def test_no_rows_and_nothing_to_do():
    x = torch.randn(3, 100).cuda()
    assert torch.equal(gs.adjust_logits(x), x) and gs.adjust_logits(x).data_ptr() != x.data_ptr()
    assert gs.adjust_logits(x[:0], allowed=torch.zeros(0, 4, dtype=torch.int32).cuda()).shape == (0, 100)
    assert torch.equal(gs.adjust_logits_backward(x, None), x)


def test_offsets_beyond_32_bits():
    rows, vocab = 20000, 120000
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    history = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    history[-1] = vocab - 1
    allowed = torch.full((rows, vocab // 32), -1, dtype=torch.int32, device="cuda")
    allowed[-2, -1] = 0x7FFFFFFF
    one = torch.ones(rows, device="cuda")
    gs.adjust_logits(x, history=history, presence=one, frequency=one, allowed=allowed, out=x)
    assert float(x[-1, -1]) == -3.0 and bool(x[-2, -1].isneginf()) and int((x != 0).sum()) == 2
    y = gs.adjust_logits(x, history=history, presence=one)
    assert float(y[-1, -1]) == -4.0 and bool(y[-2, -1].isneginf()) and int((y != 0).sum()) == 2


def test_gradient_is_the_differences():
    """Away from 0 the adjusted logits are linear in each logit: differences of the 64-bit form are the gradient."""
    x, how, allowed = inputs(3, 400, 100, 10, True)
    x = torch.where(x.abs() < 0.01, 0.5, x)
    h = 1e-3
    up, down = (adjust64(x.double().add(s).float(), **how, allowed=allowed)[0] for s in (h, -h))
    step = (x.double().add(h).float().double() - x.double().add(-h).float().double())
    want = torch.where(allowed, (up - down) / step, 0.0)
    got = back(torch.ones(3, 400).cuda(), x.cuda(), how, allowed).double().cpu()
    assert float((got - want).abs().max()) < 1e-6      # 64-bit differences of numbers below 20 over 2e-3, and 2 roundings


@pytest.mark.parametrize("dtype", DTYPES)
def test_autograd(dtype):
    x, how, allowed = inputs(4, 700, 60, 5, True, dtype)
    leaf = x.cuda().requires_grad_()
    out = call(leaf, how, allowed)
    assert torch.equal(out, call(x.cuda(), how, allowed))
    d = torch.randn_like(out)
    out.backward(d)
    assert torch.equal(leaf.grad, back(d, x.cuda(), how, allowed))
    for less in (("history",), ("history", "repetition"), ()):
        leaf.grad = None
        part = {k: v for k, v in how.items() if k in less}
        call(leaf, part, allowed).sum().backward()      # an expanded gradient
        assert torch.equal(leaf.grad, back(torch.ones_like(out), x.cuda(), part, allowed))
    y = leaf * 1.0
    out = call(y, how, allowed)
    with torch.no_grad():
        call(y, how, allowed, out=y)
    with pytest.raises(RuntimeError, match="modified"):
        out.sum().backward()


def test_what_has_no_gradient_says_so():
    x, how, _ = inputs(4, 700, 60, 5, False)
    xs = x.cuda().requires_grad_()
    with pytest.raises(RuntimeError, match="out"):
        call(xs, how, None, out=torch.empty_like(xs))
    for name in ("repetition", "presence", "frequency", "bias"):
        with pytest.raises(RuntimeError, match="no gradient"):
            gs.adjust_logits(x.cuda(), **{k: v.cuda().requires_grad_(k == name) for k, v in how.items()})
    with torch.no_grad():
        gs.adjust_logits(xs, **{k: v.cuda().requires_grad_(k == "bias") for k, v in how.items()})
    with pytest.raises(RuntimeError):
        torch.vmap(lambda a: gs.adjust_logits(a))(torch.zeros(2, 3, 40, device="cuda"))


def test_refusals():
    x, how, allowed = inputs(4, 100, 8, 3, True)
    x, allowed = x.cuda(), pack(allowed).cuda()
    how = {k: v.cuda() for k, v in how.items()}

    def calls(kind, *changes):
        for c in changes:
            with pytest.raises(kind):
                gs.adjust_logits(**{"logits": x, **how, "allowed": allowed, **c})

    calls(TypeError, dict(logits=x.double()), dict(history=how["history"].float()), dict(prompt=how["prompt"].long()), dict(repetition=1.2),
          dict(bias=how["bias"].half()), dict(allowed=allowed.bool()), dict(bias_tokens=how["bias"]))
    calls(ValueError, dict(logits=x.cpu()), dict(logits=x[0]), dict(logits=x.t()), dict(history=how["history"][:3]), dict(history=how["history"][0]),
          dict(history=how["history"].cpu()), dict(history=None), dict(prompt=how["prompt"][:3]), dict(repetition=how["repetition"].unsqueeze(1)),
          dict(bias=None), dict(bias_tokens=None), dict(bias=how["bias"][:, :2]), dict(allowed=allowed[:, :3]), dict(allowed=allowed.cpu()),
          dict(out=x[:3]), dict(out=x.half()), dict(out=torch.empty(100, 4, device="cuda").t()))
    calls(gs.GsortError, dict(out=torch.empty(500, device="cuda").as_strided((4, 100), (50, 1))))
    buffer = torch.zeros(5, 100, device="cuda")
    with pytest.raises(gs.GsortError):
        gs.adjust_logits(buffer[:4], out=buffer[1:])
    with pytest.raises(ValueError, match="logits"):
        gs.adjust_logits_backward(x, None, history=how["history"], repetition=how["repetition"])
    with pytest.raises(gs.GsortError):
        gs.adjust_logits_backward(x.clone(), x, history=how["history"], repetition=how["repetition"], out=x)


def test_an_output_in_a_graph_is_refused():
    """It would keep its node, whose gradient knows nothing of the adjustments; under no_grad() it is the caller's to say so."""
    x, how, allowed = inputs(4, 700, 60, 5, True)
    leaf = x.cuda().requires_grad_()
    y = leaf * 1.0
    before = y.detach().clone()
    for out in (y, leaf):
        with pytest.raises(RuntimeError, match="no gradient"):
            call(out.detach(), how, allowed, out=out)
        with pytest.raises(RuntimeError, match="no gradient"):
            back(torch.ones_like(before), x.cuda(), how, allowed, out=out)
        with pytest.raises(RuntimeError, match="no gradient"):
            gs.embed_tokens_backward(torch.ones(9, 700, device="cuda"), torch.zeros(9, dtype=torch.int64, device="cuda"), 4, out=out)
    assert torch.equal(y, before) and torch.equal(leaf, before)
    with torch.no_grad():
        assert call(y, how, allowed, out=y) is y and torch.equal(y, call(before, how, allowed))
