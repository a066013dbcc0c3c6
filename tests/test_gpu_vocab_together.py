"""Embedding, adjusted logits, clipped gradients and the operators that were there, as a
user's steps call them: a training step and a decode step, in CUDA graphs, on side
streams, with nothing held afterwards."""
import gc
import importlib.util
import os

import pytest
import torch

import bitonic_networks_gb300 as gs
from conftest import ROOT
from vocab_ref import pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def step_of(model, tokens, targets, allowed=None, history=None, repetition=None):
    """Loss of a model with a shared table: the head is the table, so its gradient has two parts."""
    x = gs.embed_tokens(model["table"], tokens, scale=model["scale"])
    logits = x @ model["table"].t()
    logits = gs.adjust_logits(logits, history=history, repetition=repetition, allowed=allowed)
    r = gs.token_logprobs(logits, targets)
    return -r.logprobs.sum()


def test_a_training_step_with_a_shared_table():
    g = torch.Generator(device="cuda").manual_seed(5)
    vocab, width, n = 300, 64, 500
    table = (torch.randn(vocab, width, generator=g, device="cuda") * 0.3).requires_grad_()
    tokens, targets = torch.randint(vocab, (2, n), generator=g, device="cuda")
    tokens[:20] = -1
    history = torch.randint(vocab, (n, 9), generator=g, device="cuda")
    repetition = torch.rand(n, generator=g, device="cuda") + 0.5
    allowed = torch.rand(n, vocab, generator=g, device="cuda") < 0.7
    allowed[torch.arange(n), targets] = True
    words = pack(allowed).cuda()
    step_of(dict(table=table, scale=2.0), tokens, targets, words, history, repetition).backward()

    t = table.detach().double().requires_grad_()
    x = torch.where((tokens >= 0).unsqueeze(1), t[tokens.clamp(min=0)] * 2.0, 0.0)
    y = x @ t.t()
    seen = torch.zeros_like(y, dtype=torch.bool).scatter_(1, history, True)
    r = repetition.double().unsqueeze(1)
    y = torch.where(seen, torch.where(y > 0, y / r, y * r), y).masked_fill(~allowed, float("-inf"))
    (-torch.log_softmax(y, 1).gather(1, targets.unsqueeze(1)).sum()).backward()
    far = (table.grad.double() - t.grad).norm() / t.grad.norm()
    assert float(far) < 1e-4            # 32-bit products of 64 and 500 terms (signs of logits near 0 may differ)

    norm = float(t.grad.norm())
    clipped = gs.clip_gradients([table.grad], norm / 2, out=[table.grad])
    assert abs(float(clipped.norm) / norm - 1) < 1e-4 and abs(float(gs.gradient_norm([table.grad])) / norm - 0.5) < 1e-4


def test_decoding(example):
    """The example's decoding against the same in plain torch."""
    torch.manual_seed(6)
    model = example.Model(200, 64, 8, 2).cuda()
    tokens = torch.randint(200, (5,), device="cuda")
    allowed = torch.rand(5, 200, device="cuda") < 0.5
    with torch.no_grad():
        got = example.decode(model, tokens, 6, allowed=pack(allowed).cuda(), penalty=2.0)
        last, count = tokens, torch.zeros(5, 200, device="cuda")
        for i in range(6):
            y = (model.logits(last) - 2.0 * count).masked_fill(~allowed, float("-inf"))
            last = y.argmax(1)
            assert torch.equal(last, got[:, i])
            count[torch.arange(5), last] += 1


@pytest.mark.parametrize("n", [5, 3000, 9000, 70001])
def test_steps_in_cuda_graphs(n):
    """A forward and backward pass and clipping, captured on a side stream and replayed on new
    inputs, beside an eager pass; two graphs captured into one pool replay one after another."""
    g = torch.Generator(device="cuda").manual_seed(n)
    vocab, width = 700, 72
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    d, logits = torch.empty(n, width, dtype=torch.bfloat16, device="cuda"), torch.empty(n, vocab, dtype=torch.bfloat16, device="cuda")
    tokens, history = torch.empty(n, dtype=torch.int64, device="cuda"), torch.empty(n, 12, dtype=torch.int64, device="cuda")
    one = torch.ones(n, device="cuda") * 1.5
    words = torch.empty(n, (vocab + 31) // 32, dtype=torch.int32, device="cuda")

    def fill():
        for t in (table, d, logits):
            t.normal_(generator=g)
        for t in (tokens, history):
            t.random_(-3, vocab + 3, generator=g)
        words.random_(-2 ** 31, 2 ** 31 - 1, generator=g)

    def training():
        out = gs.embed_tokens(table, tokens, scale=3.0)
        d_table = gs.embed_tokens_backward(d, tokens, vocab, scale=3.0)
        d_logits = gs.adjust_logits_backward(logits, logits, history=history, repetition=one, allowed=words)
        return [out, *gs.clip_gradients([d_table, d_logits], 2.0).gradients, gs.gradient_norm([d_table, d_logits])]

    def answers():
        y = gs.adjust_logits(logits, history=history, repetition=one, frequency=one, allowed=words)
        return [y, *gs.token_logprobs(y, top=3)[1:4]]

    fill()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        training(), answers()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [], []
    for step in (training, answers):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side, pool=graphs[0].pool() if graphs else None):
            held.append(step())
        graphs.append(graph)
    for _ in range(3):
        fill()
        for graph, step, kept in zip(graphs, (training, answers), held):
            graph.replay()
            for got, want in zip(kept, step()):
                assert torch.equal(got.reshape(-1).view(torch.uint8), want.reshape(-1).view(torch.uint8))


def test_autograd_in_a_cuda_graph():
    """A whole training step under autograd, captured after its warm-up passes were dropped."""
    g = torch.Generator(device="cuda").manual_seed(8)
    table = (torch.randn(300, 64, generator=g, device="cuda") * 0.3).requires_grad_()
    tokens, targets = torch.randint(300, (2, 400), generator=g, device="cuda")
    words = torch.full((400, 10), -1, dtype=torch.int32, device="cuda")

    def step():
        gradient, = torch.autograd.grad(step_of(dict(table=table, scale=1.0), tokens, targets, words), table)
        return gs.clip_gradients([gradient], 0.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in range(3):
        tokens.random_(-1, 300, generator=g)
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        # the products of the head may be cut differently in a graph
        assert torch.allclose(held.gradients[0], want.gradients[0], rtol=1e-4, atol=1e-6) and torch.allclose(held.norm, want.norm, rtol=1e-4)


def test_every_call_runs_on_the_current_stream():
    """The inputs are filled on a side stream after work of some milliseconds: a
    launch on another stream would find them empty."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    real = [torch.randn(300, 136, generator=gen, device="cuda"), torch.randn(9000, 136, generator=gen, device="cuda"),
            torch.randn(700, 5000, generator=gen, device="cuda"), torch.randint(300, (9000,), generator=gen, device="cuda"),
            torch.randint(5000, (700, 20), generator=gen, device="cuda"), torch.randint(-99, 99, (700, 157), generator=gen, device="cuda").int(),
            torch.rand(700, generator=gen, device="cuda") + 0.5]
    late = [torch.zeros_like(t) for t in real]

    def calls(table, d, logits, tokens, history, words, r):
        yield [gs.embed_tokens(table, tokens)]
        yield [gs.embed_tokens_backward(d, tokens, 300)]
        yield [gs.embed_tokens_backward(d[:500], tokens[:500], 300)]
        y = gs.adjust_logits(logits, history=history, repetition=r, presence=r, bias_tokens=history[:, :4].contiguous(), bias=logits[:, :4].contiguous(), allowed=words)
        yield [y]
        yield [gs.adjust_logits_backward(logits, logits, history=history, repetition=r, allowed=words)]
        yield [gs.gradient_norm([d, logits])]
        clipped = gs.clip_gradients([d, logits], 1.0)
        yield [*clipped.gradients, clipped.norm]

    want = list(calls(*real))
    list(calls(*late))                          # the kernels are loaded
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(60):
            big.add_(1.0)
        filled = torch.cuda.Event()
        for to, t in zip(late, real):
            to.copy_(t)
        filled.record()
        got = list(calls(*late))
        early = not filled.query()              # every call was made before the inputs were there
        same = [torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w)]
    torch.cuda.synchronize()
    assert early and all(same), (early, same)


def test_two_calls_at_once():
    """Calls on two streams have workspaces of their own."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    d = torch.randn(20000, 256, generator=gen, device="cuda")
    tokens = [torch.randint(v, (20000,), generator=gen, device="cuda") for v in (100, 5000)]
    want = [gs.embed_tokens_backward(d, t, 5000) for t in tokens] + [gs.gradient_norm([d]), gs.gradient_norm([d[:9000].contiguous()])]
    other = d[:9000].contiguous()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((gs.embed_tokens_backward(d, tokens[i], 5000), gs.gradient_norm([d if i == 0 else other])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i]) and torch.equal(n, want[2 + i]) for i in range(2) for a, n in got[i])


def test_steps_leave_nothing_behind():
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(300, 64, generator=gen, device="cuda").requires_grad_()
    tokens, targets = torch.randint(300, (2, 400), generator=gen, device="cuda")

    def steps(count):
        for _ in range(count):
            step_of(dict(table=table, scale=1.0), tokens, targets).backward()
            gs.clip_gradients([table.grad], 1.0, out=[table.grad])
            table.grad = None
        gc.collect()
        return torch.cuda.memory_allocated()

    assert steps(3) == steps(20)
