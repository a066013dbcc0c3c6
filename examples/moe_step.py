"""A tiny mixture-of-experts language model with the library's operators, trained
for some steps and then asked for likely next tokens.

    python examples/moe_step.py [--steps N] [--tokens T] [--width H] [--experts E] [--vocab V]

Each step routes the tokens' rows to experts (route_experts), groups them by
expert (group_by_expert), moves them there (dispatch_rows), applies each
expert's matrix to its segment of the grouped layout, moves the results back
(combine_rows) and scores the given tokens (token_logprobs); the gradients go
the same way back.  The matrix products are torch's.  Prints the loss before
and after, and the alternatives to one answer with their log probabilities.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitonic_networks_gb300 as gs


class Route(torch.autograd.Function):
    """Weights (with a gradient) and experts of the k best experts of each token."""

    @staticmethod
    def forward(ctx, logits, k, how):
        weights, experts = gs.route_experts(logits, k, **how)
        ctx.save_for_backward(logits, experts)
        ctx.how = how
        ctx.mark_non_differentiable(experts)
        return weights, experts

    @staticmethod
    def backward(ctx, d_weights, _):
        logits, experts = ctx.saved_tensors
        how = {k: v for k, v in ctx.how.items() if k in ("score", "renormalise", "scale")}
        return gs.route_experts_backward(d_weights.contiguous(), logits, experts, **how), None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, groups):
        ctx.save_for_backward(*groups)
        return gs.dispatch_rows(x, groups)

    @staticmethod
    def backward(ctx, d):
        return gs.combine_rows(d.contiguous(), gs.ExpertGroups(*ctx.saved_tensors)), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, groups):
        ctx.save_for_backward(y, weights, *groups)
        return gs.combine_rows(y, groups, weights)

    @staticmethod
    def backward(ctx, d):
        y, weights, *groups = ctx.saved_tensors
        d_y, d_weights = gs.combine_rows_backward(d.contiguous(), y, gs.ExpertGroups(*groups), weights)
        return d_y, d_weights, None


class TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets):
        r = gs.token_logprobs(logits, targets)
        # an output kept as an attribute would hold its own node, and all before it, for ever
        ctx.save_for_backward(logits, targets, r.entropy, r.stats)
        return r.logprobs, r.entropy

    @staticmethod
    def backward(ctx, d_logprobs, d_entropy):
        logits, targets, entropy, stats = ctx.saved_tensors
        r = gs.TokenLogprobs(None, entropy, None, None, stats)
        return gs.token_logprobs_backward(d_logprobs.contiguous(), d_entropy.contiguous(), logits, targets, r), None


class Model(torch.nn.Module):
    def __init__(self, vocab, width, experts, k, align=16):
        super().__init__()
        self.k, self.experts, self.align = k, experts, align
        self.embed = torch.nn.Parameter(torch.randn(vocab, width) * 0.5)
        self.router = torch.nn.Parameter(torch.randn(width, experts) * width ** -0.5)
        self.expert = torch.nn.Parameter(torch.randn(experts, width, width) * width ** -0.5)
        self.head = torch.nn.Parameter(torch.randn(width, vocab) * width ** -0.5)
        self.register_buffer("bias", torch.zeros(experts))      # of the choice, moved against the load

    def logits(self, tokens):
        x = self.embed[tokens]
        how = dict(score="sigmoid", bias=self.bias, renormalise=True)
        weights, experts = Route.apply(x @ self.router, self.k, how)
        groups = gs.group_by_expert(experts, self.experts, align=self.align)
        self.load = groups.counts
        rows = Dispatch.apply(x, groups)
        starts = groups.offsets.tolist()
        out = [torch.relu(rows[a:b] @ w) for w, a, b in zip(self.expert, starts, starts[1:])]
        y = torch.cat(out + [rows.new_zeros(rows.shape[0] - starts[-1], rows.shape[1])])
        return (x + Combine.apply(y, weights, groups)) @ self.head

    def balance(self, rate=0.01):
        """Raises the choice bias of experts with less than the mean load, lowers the others'."""
        self.bias += rate * torch.sign(self.load.float().mean() - self.load.float())


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("steps", 40), ("tokens", 512), ("width", 128), ("experts", 16), ("vocab", 1000), ("k", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    model = Model(a.vocab, a.width, a.experts, a.k).cuda()
    optimiser = torch.optim.Adam(model.parameters(), lr=1e-2)
    follows = torch.randperm(a.vocab, device="cuda")            # what the model has to learn
    tokens = torch.randint(a.vocab, (a.tokens,), device="cuda")
    losses = []
    for step in range(a.steps):
        logprobs, entropy = TokenLogprobs.apply(model.logits(tokens), follows[tokens])
        loss = -logprobs.mean() - 1e-3 * entropy.mean()
        optimiser.zero_grad()
        loss.backward()
        optimiser.step()
        model.balance()
        losses.append(float(-logprobs.detach().mean()))
    print(f"negative log probability: {losses[0]:.3f} before, {losses[-1]:.3f} after {a.steps} steps")

    with torch.no_grad():                                       # one token decoded, with alternatives
        r = gs.token_logprobs(model.logits(tokens[:1]), top=5)
    print("after token", int(tokens[0]), "(given", int(follows[tokens[0]]), "in training):",
          ", ".join(f"{i}: {v:.2f}" for i, v in zip(r.top_ids[0].tolist(), r.top_logprobs[0].tolist())))
    return losses, int(r.top_ids[0, 0]), int(follows[tokens[0]])


if __name__ == "__main__":
    main()
