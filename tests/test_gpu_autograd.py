"""The operators under autograd: gradients of the public calls are those of the
backward calls, and what has no gradient says so."""
import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES

pytestmark = pytest.mark.gpu


def leaf(*shape, dtype=torch.float32, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda().requires_grad_()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score,renormalise", [("softmax", False), ("sigmoid", True)])
def test_routing(dtype, score, renormalise):
    x, bias, d = leaf(70, 24, dtype=dtype), leaf(24, seed=1), torch.randn(70, 3).cuda()
    how = dict(score=score, renormalise=renormalise, scale=1.5)
    w, e = gs.route_experts(x, 3, bias=bias, groups=4, groups_kept=2, **how)
    w0, e0 = gs.route_experts(x.detach(), 3, bias=bias.detach(), groups=4, groups_kept=2, **how)
    assert torch.equal(w, w0) and torch.equal(e, e0) and not e.requires_grad and not w0.requires_grad
    (w * d).sum().backward()
    assert torch.equal(x.grad, gs.route_experts_backward(d, x.detach(), e, **how)) and bias.grad is None


@pytest.mark.parametrize("dtype", DTYPES)
def test_row_moves(dtype):
    _, e = gs.route_experts(torch.randn(50, 8).cuda(), 2)
    g = gs.group_by_expert(e, 8, align=4)
    x, y, w = leaf(50, 40, dtype=dtype), leaf(g.rows.numel(), 40, dtype=dtype, seed=1), leaf(50, 2, seed=2)
    rows = gs.dispatch_rows(x, g)
    d = torch.randn_like(rows)
    rows.backward(d)
    assert torch.equal(x.grad, gs.combine_rows(d, g))
    for weights in (w, None):
        y.grad = None
        out = gs.combine_rows(y, g, weights)
        d = torch.randn_like(out)
        out.backward(d)
        if weights is None:
            assert torch.equal(y.grad, gs.dispatch_rows(d, g))
        else:
            d_y, d_w = gs.combine_rows_backward(d, y.detach(), g, w.detach())
            assert torch.equal(y.grad, d_y) and torch.equal(w.grad, d_w)
    # one of the two alone
    w.grad = y.grad = None
    gs.combine_rows(y.detach(), g, w).sum().backward()
    assert w.grad is not None and y.grad is None
    gs.combine_rows(y, g, w.detach()).sum().backward()          # an expanded gradient
    assert y.grad is not None


@pytest.mark.parametrize("dtype", DTYPES)
def test_log_probabilities(dtype):
    x, t = leaf(9, 300, dtype=dtype), torch.arange(9).cuda()
    plain = x.detach()
    a, b = torch.randn(9).cuda(), torch.randn(9).cuda()
    for use_lp, use_h in ((True, True), (True, False), (False, True)):
        x.grad = None
        r = gs.token_logprobs(x, t, top=4)
        r0 = gs.token_logprobs(plain, t, top=4)
        assert all(torch.equal(p, q) for p, q in zip(r, r0))
        loss = (r.logprobs * a).sum() if use_lp else 0.0
        loss = loss + (r.entropy * b).sum() if use_h else loss
        loss.backward()
        assert torch.equal(x.grad, gs.token_logprobs_backward(a if use_lp else None, b if use_h else None, plain, t, r0))
    x.grad = None
    gs.token_logprobs(x).entropy.sum().backward()
    assert x.grad is not None


def test_what_has_no_gradient_says_so():
    x = leaf(9, 300)
    with pytest.raises(RuntimeError, match="top_logprobs"):
        gs.token_logprobs(x, top=4).top_logprobs.sum().backward()
    r = gs.token_logprobs(x, top=4)
    assert not r.top_ids.requires_grad and not r.stats.requires_grad
    h = torch.autograd.grad(r.entropy.sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError):          # no second derivative
        h.sum().backward()
    x.grad = None
    with torch.no_grad():
        assert not gs.token_logprobs(x).entropy.requires_grad and not gs.route_experts(x, 2)[0].requires_grad
    changed = leaf(9, 300)
    y = changed * 1.0
    r = gs.token_logprobs(y)
    y.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        r.entropy.sum().backward()


def test_a_chain_of_calls_leaves_nothing_behind():
    x, logits, t = leaf(64, 40), leaf(64, 8, seed=1), torch.arange(64).cuda() % 40

    def steps(n):
        for _ in range(n):
            w, e = gs.route_experts(logits, 2, renormalise=True)
            g = gs.group_by_expert(e, 8)
            r = gs.token_logprobs(gs.combine_rows(gs.dispatch_rows(x, g) * 2.0, g, w), t)
            (r.logprobs.sum() + r.entropy.sum()).backward()
            x.grad = logits.grad = None
        del w, e, g, r
        return torch.cuda.memory_allocated()

    assert steps(3) == steps(20)


def test_other_kinds_of_derivatives_are_refused():
    x = torch.randn(3, 9, 40).cuda()
    with pytest.raises(RuntimeError):
        torch.vmap(lambda a: gs.token_logprobs(a).entropy)(x)
    with pytest.raises(RuntimeError):
        torch.vmap(lambda a: gs.route_experts(a, 2)[0])(x.requires_grad_())


def test_a_gradient_over_saved_logits_is_noticed():
    """Written over the logits, the gradient is no longer what the graph saved."""
    x, d = leaf(9, 300), torch.ones(9).cuda()
    y = x * 1.0
    r = gs.token_logprobs(y)
    with torch.inference_mode():
        z = x.clone()
        gs.token_logprobs_backward(None, d, z, None, gs.token_logprobs(z), out=z)
    with torch.no_grad():
        gs.token_logprobs_backward(None, d, y, None, r, out=y)
    with pytest.raises(RuntimeError, match="modified"):
        r.entropy.sum().backward()
