"""A tiny mixture-of-experts language model with the library's operators, trained
for some steps and then asked for likely next tokens.

    python examples/moe_step.py [--steps N] [--tokens T] [--width H] [--experts E] [--vocab V]

Each step routes the tokens' rows to experts (route_experts), groups them by
expert (group_by_expert), moves them there (dispatch_rows), applies each
expert's matrix to its segment of the grouped layout, moves the results back
(combine_rows) and scores the given tokens (token_logprobs); autograd takes the
gradients the same way back.  The matrix products are torch's.  Prints the loss before
and after, and the alternatives to one answer with their log probabilities.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bitonic_networks_gb300 as gs


class TokenLogprobs:
    @staticmethod
    def apply(logits, targets):
        """Log probabilities of the targets and the rows' entropies, both with gradients."""
        r = gs.token_logprobs(logits, targets)
        return r.logprobs, r.entropy


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
        weights, experts = gs.route_experts(x @ self.router, self.k, score="sigmoid", bias=self.bias, renormalise=True)
        groups = gs.group_by_expert(experts, self.experts, align=self.align)
        self.load = groups.counts
        rows = gs.dispatch_rows(x, groups)
        starts = groups.offsets.tolist()
        out = [torch.relu(rows[a:b] @ w) for w, a, b in zip(self.expert, starts, starts[1:])]
        y = torch.cat(out + [rows.new_zeros(rows.shape[0] - starts[-1], rows.shape[1])])
        return (x + gs.combine_rows(y, groups, weights)) @ self.head

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
