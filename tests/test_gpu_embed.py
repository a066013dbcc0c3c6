"""embed_tokens and its gradient against 64-bit forms: sizes, runs of equal tokens
around the pieces' ends, what is no token, strides, accumulation, order."""
import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES, strided
from vocab_ref import embed64, embed_backward64, near

pytestmark = pytest.mark.gpu


def normal(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def tokens_of(n, vocab, seed=0, dtype=torch.int64):
    """A text's: few frequent ones, many rare ones, some that are no tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = ((vocab + 1.0) ** u).long().clamp(1, vocab) - 1
    out = torch.rand(n, generator=g, device="cuda")
    t = torch.where(out < 0.05, -1, torch.where(out < 0.08, vocab, torch.where(out < 0.1, 2 ** 31 - 1, t)))
    return t.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", [(1, 1, 1), (1, 5, 8), (3, 2, 7), (17, 100, 33), (64, 1000, 64), (1000, 50, 1001), (33, 7, 4096),
                                           (5, 3, 20000)])
@pytest.mark.parametrize("scale", [1.0, 31.6])
def test_lookup(dtype, n, vocab, width, scale):
    table, tokens = normal(vocab, width, dtype=dtype), tokens_of(n, vocab, dtype=torch.int32)
    got = gs.embed_tokens(table, tokens, scale=scale)
    assert got.dtype == dtype and got.shape == (n, width) and got.is_contiguous()
    near(got, *embed64(table, tokens, scale))
    if scale == 1.0:
        held = (tokens >= 0) & (tokens < vocab)
        assert torch.equal(got[held], table[tokens[held].long()])
    for pad, off in ((8, 0), (5, 3)):
        assert torch.equal(gs.embed_tokens(strided(table, pad, off), tokens.long(), scale=scale), got)


def test_lookup_keeps_what_is_in_the_table():
    """NaN, infinities, zeros' signs and subnormals are copied; a row of NaN beside it changes nothing."""
    table = torch.tensor([[float("nan")] * 40, [float("inf"), -0.0, 1e-45, -float("inf")] * 10, [1.0] * 40]).cuda()
    for dtype in DTYPES:
        t = table.to(dtype)
        got = gs.embed_tokens(t, torch.tensor([1, 2, 7, 0], device="cuda"))
        assert torch.equal(got[:2].view(torch.uint8), t[1:].view(torch.uint8)) and bool((got[2] == 0).all()) and bool(got[3].isnan().all())


@pytest.mark.parametrize("shape", [(), (0,), (6,), (2, 3), (2, 0, 3), (2, 3, 2)])
def test_tokens_of_any_shape(shape):
    table = normal(11, 24)
    tokens = torch.randint(11, shape, device="cuda")
    out = gs.embed_tokens(table, tokens, scale=2.0)
    assert torch.equal(out, table[tokens] * 2.0)
    d = torch.randn_like(out)
    near(gs.embed_tokens_backward(d, tokens, 11, scale=2.0), *embed_backward64(d, tokens, 11, 2.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", [(0, 7, 24), (1, 1, 1), (2, 1, 8), (31, 3, 7), (64, 1000, 64), (257, 40, 33), (1000, 300, 1001),
                                           (4099, 5000, 520), (8192, 9001, 40), (8193, 9001, 40), (70001, 100, 48), (300000, 70000, 8)])
def test_gradient(dtype, n, vocab, width):
    d, tokens = normal(n, width, dtype=dtype), tokens_of(n, vocab)
    want = embed_backward64(d, tokens, vocab, 1.5)
    got = gs.embed_tokens_backward(d, tokens, vocab, scale=1.5)
    assert got.dtype == dtype and got.shape == (vocab, width)
    near(got, *want)
    assert torch.equal(got, gs.embed_tokens_backward(d, tokens.int(), vocab, scale=1.5))        # the same order of sums
    if n:
        near(gs.embed_tokens_backward(strided(d, 5, 3), tokens, vocab, scale=1.5), *want)
        out = strided(torch.full_like(got, 7.0), 3, 1)
        assert gs.embed_tokens_backward(d, tokens, vocab, scale=1.5, out=out) is out
        near(out, *want)
        buffer = out.as_strided((vocab, width + 3), (width + 3, 1))[: vocab - 1 or 1, width:]
        assert vocab == 1 or bool(buffer.isnan().all())        # between the rows nothing is written


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [16, 64, 300, 1024])
@pytest.mark.parametrize("lengths", [[1000], [8191, 1], [1, 8191], [31, 33, 32, 64, 1, 255, 257, 256, 512, 513, 1023], [63, 65, 64, 7, 1, 1, 9, 3000, 5, 2000],
                                     [20000, 3, 1, 50000], [256] * 40, [8] * 200, [1] * 3000])
def test_runs_of_equal_tokens(dtype, width, lengths):
    """Runs that begin and end at, before and behind the ends of the pieces."""
    tokens = torch.cat([torch.full((m,), 3 * i + 1) for i, m in enumerate(lengths)])
    tokens = tokens[torch.randperm(tokens.numel(), generator=torch.Generator().manual_seed(1))].cuda()
    d, vocab = normal(tokens.numel(), width, dtype=dtype), 3 * len(lengths) + 5
    near(gs.embed_tokens_backward(d, tokens, vocab), *embed_backward64(d, tokens, vocab, 1.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [40, 8193])
def test_nothing_but_padding(dtype, n):
    d = torch.full((n, 72), float("nan"), dtype=dtype, device="cuda")
    for t in (-1, 50, 2 ** 40, -2 ** 63):
        tokens = torch.full((n,), t, device="cuda")
        assert torch.equal(gs.embed_tokens_backward(d, tokens, 50), torch.zeros(50, 72, dtype=dtype, device="cuda"))
        assert torch.equal(gs.embed_tokens(d[:50], tokens), torch.zeros(n, 72, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("width", [64, 1001])
def test_nan_and_infinities_stay_in_their_rows(width):
    n, vocab = 3000, 40
    d, tokens = normal(n, width), torch.arange(n, device="cuda") % vocab
    clean = gs.embed_tokens_backward(d, tokens, vocab)
    d[5], d[17] = float("nan"), float("inf")
    got = gs.embed_tokens_backward(d, tokens, vocab)
    others = [v for v in range(vocab) if v not in (5, 17)]
    assert bool(got[5].isnan().all()) and bool(got[17].isposinf().all()) and torch.equal(got[others], clean[others])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", [(0, 5, 16), (1, 5, 16), (700, 90, 33), (9000, 300, 64)])
def test_accumulated(dtype, n, vocab, width):
    d, tokens, old = normal(n, width, dtype=dtype), tokens_of(n, vocab), normal(vocab, width, dtype=dtype, seed=1)
    want = embed_backward64(d, tokens, vocab, 0.5, old)
    for out in (old.clone(), strided(old, 3, 1)):
        assert gs.embed_tokens_backward(d, tokens, vocab, scale=0.5, out=out, accumulate=True) is out
        near(out, *want)
        held = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        held[tokens[(tokens >= 0) & (tokens < vocab)]] = True
        assert torch.equal(out[~held], old[~held])


def test_rows_of_the_last_sequence_only():
    """Tokens behind the sequences' ends are padding: their gradients, whatever they hold, go nowhere."""
    d, tokens = normal(4, 50, 32), torch.randint(9, (4, 50), device="cuda")
    tokens[:, 30:] = -1
    d[:, 30:] = float("nan")
    near(gs.embed_tokens_backward(d, tokens, 9), *embed_backward64(d[:, :30], tokens[:, :30], 9, 1.0))


def test_given_workspace():
    d, tokens = normal(9000, 64), tokens_of(9000, 500)
    need = gs.embed_workspace_bytes(9000, 500, 64, torch.float32)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = gs.embed_tokens_backward(d, tokens, 500)
    for _ in range(2):
        assert torch.equal(gs.embed_tokens_backward(d, tokens, 500, workspace=ws), want)
    with pytest.raises(gs.GsortError, match="WORKSPACE"):
        gs.embed_tokens_backward(d, tokens, 500, workspace=ws[:-1])


def test_offsets_beyond_32_bits():
    vocab, width = 270000, 8192
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    assert table.numel() > 2 ** 31
    last = torch.tensor([vocab - 1, 3, vocab - 2, vocab - 1], device="cuda")
    table[vocab - 1], table[vocab - 2], table[3] = 3.0, 2.0, 1.0
    assert gs.embed_tokens(table, last)[:, ::1000].tolist() == [[x] * 9 for x in (3.0, 1.0, 2.0, 3.0)]
    d = gs.embed_tokens_backward(torch.ones(4, width, dtype=torch.bfloat16, device="cuda"), last, vocab, out=table)
    assert float(d[vocab - 1].min()) == float(d[vocab - 1].max()) == 2.0 and float(d[vocab - 2].min()) == 1.0 == float(d[3].max())
    assert float(d.float().sum()) == 4.0 * width
    del table, d
    many = torch.zeros(265000, 8192, dtype=torch.bfloat16, device="cuda")      # more positions than fit 32 bits of elements
    many[-1] = 5.0
    tokens = torch.full((265000,), 1, device="cuda")
    tokens[-1] = 0
    d = gs.embed_tokens_backward(many, tokens, 2)
    assert bool((d[0] == 5.0).all()) and bool((d[1] == 0).all())
    out = gs.embed_tokens(d, tokens)
    assert bool((out[-1] == 5.0).all()) and float(out.float().abs().sum()) == 5.0 * 8192


def test_gradient_is_the_differences():
    """The lookup is linear in the table: <d, f(table + h) - f(table)> = <gradient, h>, in numbers that
    32 bits hold exactly."""
    g = torch.Generator(device="cuda").manual_seed(3)
    table, h = (torch.randint(-8, 9, (30, 20), generator=g, device="cuda").float() for _ in range(2))
    tokens = torch.randint(-1, 31, (500,), generator=g, device="cuda")
    d = torch.randint(-8, 9, (500, 20), generator=g, device="cuda").float()
    change = (d.double() * (gs.embed_tokens(table + h, tokens, scale=0.5) - gs.embed_tokens(table, tokens, scale=0.5)).double()).sum()
    assert float(change) == float((gs.embed_tokens_backward(d, tokens, 30, scale=0.5).double() * h.double()).sum())


@pytest.mark.parametrize("dtype", DTYPES)
def test_autograd(dtype):
    table, tokens = normal(60, 40, dtype=dtype).requires_grad_(), tokens_of(300, 60).view(3, 100)
    out = gs.embed_tokens(table, tokens, scale=2.0)
    d = torch.randn_like(out)
    out.backward(d)
    assert torch.equal(table.grad, gs.embed_tokens_backward(d, tokens, 60, scale=2.0))
    table.grad = None
    gs.embed_tokens(table, tokens).sum().backward()            # an expanded gradient
    count = torch.bincount(tokens[(tokens >= 0) & (tokens < 60)].flatten(), minlength=60)
    assert torch.equal(table.grad, count.to(dtype).unsqueeze(1).expand(-1, 40))
    with torch.no_grad():
        assert not gs.embed_tokens(table, tokens).requires_grad
    h = torch.autograd.grad(gs.embed_tokens(table, tokens).sum(), table, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        h.sum().backward()
    y = table * 1.0
    out = gs.embed_tokens(y, tokens)
    moved = tokens.clone()
    again = gs.embed_tokens(y, moved)
    moved.add_(1)
    with pytest.raises(RuntimeError, match="modified"):
        again.sum().backward()


def test_refusals():
    table, tokens = normal(9, 24), torch.zeros(5, dtype=torch.int64, device="cuda")
    d = normal(5, 24)
    for call in (lambda: gs.embed_tokens(table, tokens.float()), lambda: gs.embed_tokens(table.int(), tokens), lambda: gs.embed_tokens(table, [1]),
                 lambda: gs.embed_tokens_backward(d, tokens.short(), 9), lambda: gs.embed_tokens_backward(d, tokens, 9.5)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gs.embed_tokens(table[0], tokens), lambda: gs.embed_tokens(table.t(), tokens), lambda: gs.embed_tokens(table, tokens.cpu()),
                 lambda: gs.embed_tokens(table, torch.zeros(10, dtype=torch.int64, device="cuda")[::2]),
                 lambda: gs.embed_tokens_backward(d[:4], tokens, 9), lambda: gs.embed_tokens_backward(d, tokens, 0),
                 lambda: gs.embed_tokens_backward(d, tokens, 2 ** 40), lambda: gs.embed_tokens_backward(d, tokens, 9, accumulate=True),
                 lambda: gs.embed_tokens_backward(d, tokens, 9, out=table[:8]), lambda: gs.embed_tokens_backward(d, tokens, 9, out=table.half()),
                 lambda: gs.embed_tokens_backward(d.t().contiguous().t(), tokens, 9)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gs.embed_tokens(table, tokens, scale=float("nan")), lambda: gs.embed_tokens(normal(1, 24).expand(9, 24), tokens),
                 lambda: gs.embed_tokens_backward(d, tokens, 5, out=d), lambda: gs.embed_tokens_backward(d, tokens, 9, scale=float("inf"))):
        with pytest.raises(gs.GsortError):
            call()
