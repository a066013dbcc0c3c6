"""The example model: its whole gradient against the same model in plain 64-bit
torch, and that it learns."""
import gc
import importlib.util
import os

import pytest
import torch

import bitonic_networks_gb300 as gs
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_step", os.path.join(ROOT, "examples", "moe_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_gradients_of_the_model(example):
    torch.manual_seed(3)
    model = example.Model(200, 64, 8, 2, align=16).cuda()
    tokens, targets = torch.randint(200, (2, 97), device="cuda")
    logprobs, entropy = example.TokenLogprobs.apply(model.logits(tokens), targets)
    (-logprobs.mean() - 0.1 * entropy.mean()).backward()

    p = {k: v.detach().double().requires_grad_() for k, v in model.named_parameters()}
    x = p["embed"][tokens]
    router = x @ p["router"]
    _, chosen = gs.route_experts((x @ p["router"]).detach().float(), 2, score="sigmoid", bias=model.bias, renormalise=True)
    s = torch.sigmoid(router).gather(1, chosen.long())
    w = s / s.sum(1, keepdim=True)
    y = torch.relu(torch.einsum("th,tkho->tko", x, p["expert"][chosen.long()]))
    lp = torch.log_softmax((x + (w.unsqueeze(-1) * y).sum(1)) @ p["head"], -1)
    h = -(lp.exp() * lp).sum(-1)
    (-lp.gather(1, targets.unsqueeze(1)).mean() - 0.1 * h.mean()).backward()
    for name, v in model.named_parameters():
        far = (v.grad.double() - p[name].grad).norm() / p[name].grad.norm()
        assert far < 1e-4, (name, float(far))     # 32-bit products of 64 and 200 terms, a few in a row


def test_the_example_learns(example):
    losses, best, given = example.main(["--steps", "40", "--tokens", "256", "--vocab", "300"])
    assert losses[-1] < 0.25 * losses[0] and best == given


def test_a_layer_in_a_cuda_graph():
    """A decode step's calls captured on a side stream and replayed on new inputs
    (small and large enough for the two kernels of the grouping)."""
    for tokens in (16, 3000):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        logits, x = torch.empty(tokens, 64).cuda(), torch.empty(tokens, 200, dtype=torch.bfloat16).cuda()
        answers = torch.empty(tokens, 5000, dtype=torch.bfloat16).cuda()

        def fill():
            for t in (logits, x, answers):
                t.normal_(generator=g)

        def step():
            w, e = gs.route_experts(logits, 4, renormalise=True)
            groups = gs.group_by_expert(e, 64, align=8)
            out = gs.combine_rows(gs.dispatch_rows(x, groups), groups, w)
            r = gs.token_logprobs(answers, top=3)
            return [w, e, *groups, out, r.entropy, r.top_logprobs, r.top_ids]

        fill()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
        for _ in range(3):
            fill()
            graph.replay()
            for got, want in zip(held, step()):
                assert torch.equal(got, want)


def test_training_leaves_no_tensors_behind(example):
    """What a step holds on the device is free again after it."""
    torch.manual_seed(4)
    model = example.Model(200, 64, 8, 2).cuda()
    tokens, targets = torch.randint(200, (2, 97), device="cuda")

    def steps(count):
        for _ in range(count):
            logprobs, entropy = example.TokenLogprobs.apply(model.logits(tokens), targets)
            (-logprobs.mean() - 0.1 * entropy.mean()).backward()
            model.zero_grad()
        del logprobs, entropy
        gc.collect()
        return torch.cuda.memory_allocated()

    assert steps(3) == steps(20)


def test_every_call_runs_on_the_current_stream():
    """The inputs are filled on a side stream after work of some milliseconds: a
    launch on another stream would find them empty."""
    tokens, experts, width, vocab = 700, 64, 136, 5000
    gen = torch.Generator(device="cuda").manual_seed(1)
    real = [torch.randn(tokens, n, generator=gen, device="cuda") for n in (experts, width, vocab, 4)]
    late = [torch.zeros_like(t) for t in real]
    given = torch.arange(tokens, device="cuda") % vocab

    def calls(logits, x, answers, d):
        w, e = gs.route_experts(logits, 4, renormalise=True)
        yield [w, e]
        yield [gs.route_experts_backward(d, logits, e, renormalise=True)]
        g = gs.group_by_expert(e, experts, align=8)
        yield list(g)
        rows = gs.dispatch_rows(x, g)
        yield [rows]
        yield [gs.combine_rows(rows, g, w)]
        yield list(gs.combine_rows_backward(x, rows, g, w))
        r = gs.token_logprobs(answers, given, top=3)
        yield list(r)
        yield [gs.token_logprobs_backward(d[:, 0].contiguous(), None, answers, given, r)]

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
