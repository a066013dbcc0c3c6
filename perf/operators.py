"""Cases of the language-model operators: routing to experts, grouping by expert, moving rows to the experts and back,
and log probabilities of given tokens with entropy and top alternatives.

`run` computes them in plain torch operations, in 32 bits, or (own) with the library's calls.
"""
import math

import torch

own = False

INF = float("inf")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a few requests decode one token each: only latency counts
        dict(name="route decode", op="route", tokens=8, experts=128, k=8, dtype="bf16", score="softmax", bias=False,
             groups=1, kept=1, group_score="max", renormalise=True, scale=1.0, grad=False, padded=False),
        # a long prompt through a router with a balance bias and limited groups
        dict(name="route prefill", op="route", tokens=16384, experts=256, k=8, dtype="f32", score="sigmoid", bias=True,
             groups=8, kept=4, group_score="top2", renormalise=True, scale=2.5, grad=False, padded=False),
        # a training batch with padded tokens (rows masked whole): choice and gradient
        dict(name="route train", op="route", tokens=65536, experts=60, k=4, dtype="bf16", score="softmax", bias=False,
             groups=1, kept=1, group_score="max", renormalise=False, scale=1.0, grad=True, padded=True),
        # grouping alone: a decode batch, and a training batch padded to the tiles of the experts' products
        dict(name="group decode", op="group", tokens=64, experts=256, k=8, align=16, padded=False),
        dict(name="group train", op="group", tokens=65521, experts=128, k=8, align=128, padded=True),
        # rows to the experts and back: decode, a long prompt, a training step (all gradients) with an odd width
        dict(name="move decode", op="move", tokens=16, experts=128, k=8, width=4096, dtype="bf16", align=1,
             grad=False, padded=False),
        dict(name="move prefill", op="move", tokens=16384, experts=256, k=8, width=4096, dtype="bf16", align=16,
             grad=False, padded=False),
        dict(name="move train", op="move", tokens=8191, experts=64, k=6, width=1001, dtype="f32", align=1,
             grad=True, padded=True),
        # answers: a few rows with alternatives (some constrained to a part of the vocabulary), a serving batch,
        # scoring of a prompt on an odd vocabulary inside padded rows, and a training step
        dict(name="logprobs decode", op="logprobs", rows=4, vocab=32000, stride=32000, dtype="bf16", top=5,
             grad=False, masked=True),
        dict(name="logprobs batch", op="logprobs", rows=64, vocab=131072, stride=131072, dtype="f32", top=20,
             grad=False, masked=False),
        dict(name="logprobs score", op="logprobs", rows=4096, vocab=100003, stride=100096, dtype="bf16", top=1,
             grad=False, masked=False),
        dict(name="logprobs train", op="logprobs", rows=8192, vocab=131072, stride=131072, dtype="bf16", top=0,
             grad=True, masked=False),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["route", "group", "move", "logprobs"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    grad, padded = rng.random() < 0.4, rng.random() < 0.4
    experts = rng.choice([8, 16, 24, 32, 60, 64, 96, 100, 128, 160, 256, 384, 512])
    k = rng.randint(1, 8)
    if op == "route":
        case = dict(op=op, tokens=_log_int(rng, 1, 65536), experts=experts, k=k, dtype=dtype, grad=grad, padded=padded,
                    renormalise=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]))
        if rng.random() < 0.5:
            case.update(score="softmax", bias=False, group_score="max")
        else:
            case.update(score="sigmoid", bias=rng.random() < 0.7, group_score=rng.choice(["max", "top2"]))
        groups = rng.choice([1, 1, 2, 4, 8])
        if experts % groups or experts // groups < 4:
            groups = 1
        kept = rng.randint(max(1, -(-k * groups // experts)), groups)
        case.update(groups=groups, kept=kept)
        return case
    if op == "group":
        return dict(op=op, tokens=_log_int(rng, 1, 131072), experts=experts, k=k, align=rng.choice([1, 8, 16, 128]), padded=padded)
    if op == "move":
        width = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)])
        most = max(1, min(32768, (1 << 29) // (width * k * (4 if dtype == "f32" else 2))))
        return dict(op=op, tokens=_log_int(rng, 1, most), experts=experts, k=k, width=width, dtype=dtype,
                    align=rng.choice([1, 1, 16]), grad=grad, padded=padded)
    vocab = _log_int(rng, 1000, 200000)
    most = max(1, min(8192, (1 << 30) // (vocab * (4 if dtype == "f32" else 2))))
    return dict(op=op, rows=_log_int(rng, 1, most), vocab=vocab, stride=vocab + rng.choice([0, 0, 1, 64]), dtype=dtype,
                top=rng.choice([0, 1, 5, 20, 32]), grad=grad, masked=rng.random() < 0.3)


def _capacity(case):
    """Rows of the grouped layout: every pair, and the padding that the groups can need at most."""
    pairs, align = case["tokens"] * case["k"], case["align"]
    return (pairs + min(case["experts"], pairs) * (align - 1)) // align * align


# ------------------------------------------------------------------ inputs
def _router_logits(gen, tokens, experts):
    """What a router's product gives: experts of unequal popularity."""
    x = torch.randn(tokens, experts, generator=gen, device="cuda")
    return x.mul_(1.5).add_(torch.randn(experts, generator=gen, device="cuda").mul_(0.7))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def chance(p, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") < p

    state = {"case": case}
    if case["op"] == "logprobs":
        rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        whole = torch.empty(rows, case["stride"], dtype=dtype, device="cuda")
        whole.normal_(0.0, 2.5, generator=gen)
        logits = whole[:, :vocab]
        targets = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        # a model that has learnt something: most given tokens are likely ones
        likely = normal(rows).mul_(2.0).add_(9.0)
        at = torch.arange(rows, device="cuda")
        logits[at, targets] = torch.where(chance(0.7, rows), likely, normal(rows)).to(dtype)
        if case["masked"]:  # constrained answers: most of the vocabulary is masked in half of the rows
            mask = chance(0.5, rows, 1) & chance(0.95, rows, vocab)
            logits.masked_fill_(mask, -INF)
        if case["grad"]:  # prompt tokens carry no loss
            targets = torch.where(chance(0.1, rows), torch.full_like(targets, -1), targets)
            state.update(d_logprobs=normal(rows) / rows, d_entropy=normal(rows) / rows)
        state.update(logits=logits, targets=targets)
        return state

    tokens, experts, k = case["tokens"], case["experts"], case["k"]
    logits = _router_logits(gen, tokens, experts)
    padding = chance(0.1, tokens, 1) if case["padded"] else torch.zeros(tokens, 1, dtype=torch.bool, device="cuda")
    if case["op"] == "route":
        state["logits"] = logits.masked_fill_(padding, -INF).to(DTYPES[case["dtype"]])
        # balance biases move by a small fixed step a time
        state["bias"] = (torch.randint(-60, 61, (experts,), generator=gen, device="cuda") * 0.001) if case["bias"] else None
        if case["grad"]:
            state["d_weights"] = normal(tokens, k)
        return state
    chosen = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    state["experts"] = chosen.masked_fill_(padding, -1).contiguous()
    if case["op"] == "move":
        dtype, width = DTYPES[case["dtype"]], case["width"]
        state["weights"] = torch.softmax(normal(tokens, k), -1)
        state["x"] = normal(tokens, width).to(dtype)
        state["y"] = torch.empty(_capacity(case), width, dtype=dtype, device="cuda").normal_(generator=gen)
        if case["grad"]:
            state["d_out"] = normal(tokens, width).to(dtype)
            state["d_rows"] = torch.empty(_capacity(case), width, dtype=dtype, device="cuda").normal_(generator=gen)
    return state


# ------------------------------------------------------------- plain forms
def _scores(x, score):
    """Scores over an expert axis; experts at -inf take no part."""
    part = x > -INF
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(-1, keepdim=True)
        e = torch.exp(torch.where(part, x - top, -INF))
        s = e / e.sum(-1, keepdim=True)
    return torch.where(part, s, 0.0)


def _plain_route(case, logits, bias):
    x = logits.float()
    k, groups = case["k"], case["groups"]
    s = _scores(x, case["score"])
    value = x if bias is None else torch.where(x > -INF, s + bias, -INF)
    if groups > 1:
        by = value if case["group_score"] == "max" or bias is not None else torch.where(x > -INF, s, -INF)
        best = torch.sort(by.view(x.shape[0], groups, -1), dim=-1, descending=True).values
        first, second = best[..., 0], best[..., 1]
        if case["group_score"] == "top2":
            first = first + torch.where(second > -INF, second, 0.0)
        kept = torch.sort(first, dim=-1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros_like(first, dtype=torch.bool).scatter_(1, kept, True)
        value = torch.where(keep.repeat_interleave(x.shape[1] // groups, 1), value, -INF)
    found = torch.sort(value, dim=-1, descending=True, stable=True)
    there, at = found.values[:, :k] > -INF, found.indices[:, :k]
    w = torch.where(there, s.gather(1, at), 0.0)
    if case["renormalise"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return w * case["scale"], torch.where(there, at, -1).to(torch.int32)


def _plain_route_backward(case, d_weights, logits, experts):
    x = logits.float()
    there, at = experts >= 0, experts.clamp(min=0).long()
    s = _scores(x, case["score"])
    w = torch.where(there, s.gather(1, at), 0.0)
    d = torch.where(there, d_weights, 0.0) * case["scale"]
    if case["renormalise"]:
        total = w.sum(-1, keepdim=True)
        q = torch.where(total > 0, w / total, 0.0)
        d = torch.where(total > 0, (d - (d * q).sum(-1, keepdim=True)) / total, 0.0)
    if case["score"] == "sigmoid":
        dx = torch.zeros_like(x).scatter_add_(1, at, d * w * (1.0 - w) * there)
    else:
        dx = torch.zeros_like(x).scatter_add_(1, at, d * w * there) - s * (d * w).sum(-1, keepdim=True)
        if case["renormalise"]:  # the sum is zero but for rounding: experts that were not chosen get nothing
            dx = torch.where(torch.zeros_like(x).scatter_add_(1, at, there.float()) > 0, dx, 0.0)
    return dx.to(logits.dtype)


def _plain_group(case, experts):
    number, align = case["experts"], case["align"]
    flat = experts.reshape(-1).long()
    there = (flat >= 0) & (flat < number)
    key = torch.where(there, flat, number)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(number + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts[:number] + (align - 1)) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    first = counts.cumsum(0) - counts
    by = key[order]
    place = torch.arange(flat.numel(), device=flat.device) - first[by] + offsets[by]
    held = by < number
    positions = torch.empty_like(flat).scatter_(0, order, torch.where(held, place, -1))
    spare = _capacity(case)
    rows = torch.full((spare + 1,), -1, dtype=torch.int64, device=flat.device)
    rows.scatter_(0, torch.where(held, place, spare), torch.where(held, order, -1))
    return (offsets.to(torch.int32), counts[:number].to(torch.int32), rows[:spare].to(torch.int32),
            positions.view(experts.shape).to(torch.int32))


def _plain_dispatch(x, rows, k):
    held = (rows >= 0).unsqueeze(1)
    return torch.where(held, x[rows.clamp(min=0).long() // k], torch.zeros((), dtype=x.dtype, device=x.device))


def _plain_combine(y, positions, weights):
    held = positions >= 0
    w = held.float() if weights is None else torch.where(held, weights, 0.0)
    return (y[positions.clamp(min=0).long()].float() * w.unsqueeze(-1)).sum(1).to(y.dtype)


def _plain_combine_backward(d_out, y, rows, positions, weights):
    k = positions.shape[1]
    held, pair = (rows >= 0).unsqueeze(1), rows.clamp(min=0).long()
    d_y = torch.where(held, d_out[pair // k].float() * weights.reshape(-1)[pair].unsqueeze(1), 0.0).to(y.dtype)
    d_w = (y[positions.clamp(min=0).long()].float() * d_out.float().unsqueeze(1)).sum(-1)
    return d_y, torch.where(positions >= 0, d_w, 0.0)


def _plain_logprobs(case, logits, targets):
    x = logits.float()
    part = x > -INF
    top = x.amax(-1, keepdim=True)
    d = torch.where(part, x - top, 0.0)
    e = torch.where(part, torch.exp(d), 0.0)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    given = targets.clamp(min=0).unsqueeze(1)
    lp = torch.where(part.gather(1, given), d.gather(1, given) - log_total, -INF)
    lp = torch.where(targets.unsqueeze(1) >= 0, lp, 0.0).squeeze(1)
    entropy = torch.where(total > 0, log_total - (e * d).sum(-1, keepdim=True) / total, 0.0)
    out = {"logprobs": lp, "entropy": entropy.squeeze(1)}
    if case["top"]:
        # one whole number to a token: greater logits first, then lower indices
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        key = order * (1 << 20) + ((1 << 20) - 1 - torch.arange(x.shape[1], device=x.device))
        at = torch.topk(key, case["top"], dim=-1).indices
        held = part.gather(1, at)
        out["top_logprobs"] = torch.where(held, d.gather(1, at) - log_total, -INF)
        out["top_ids"] = torch.where(held, at, -1).to(torch.int32)
    return out, (d, e, total, log_total, entropy)


def _plain_logprobs_backward(logits, targets, sums, d_logprobs, d_entropy):
    d, e, total, log_total, entropy = sums
    p = torch.where(total > 0, e / total, 0.0)
    held = (targets >= 0).unsqueeze(1)
    g = torch.where(held, d_logprobs.unsqueeze(1), 0.0)
    dx = -p * (g + d_entropy.unsqueeze(1) * torch.where(p > 0, d - log_total + entropy, 0.0))
    dx.scatter_add_(1, targets.clamp(min=0).unsqueeze(1), torch.where(torch.isfinite(log_total), g, 0.0))
    return dx.to(logits.dtype)


# --------------------------------------------------------------------- run
def _run_plain(case, state):
    if case["op"] == "route":
        w, experts = _plain_route(case, state["logits"], state["bias"])
        out = {"weights": w, "experts": experts}
        if case["grad"]:
            out["d_logits"] = _plain_route_backward(case, state["d_weights"], state["logits"], experts)
        return out
    if case["op"] == "logprobs":
        out, sums = _plain_logprobs(case, state["logits"], state["targets"])
        if case["grad"]:
            out["d_logits"] = _plain_logprobs_backward(state["logits"], state["targets"], sums, state["d_logprobs"], state["d_entropy"])
        return out
    offsets, counts, rows, positions = _plain_group(case, state["experts"])
    if case["op"] == "group":
        return {"offsets": offsets, "counts": counts, "rows": rows, "positions": positions}
    out = {"rows": _plain_dispatch(state["x"], rows, case["k"]), "out": _plain_combine(state["y"], positions, state["weights"])}
    if case["grad"]:
        out["d_y"], out["d_weights"] = _plain_combine_backward(state["d_out"], state["y"], rows, positions, state["weights"])
        out["d_x"] = _plain_combine(state["d_rows"], positions, None)
    return out


def _run_own(case, state):
    import bitonic_networks_gb300 as gs
    if case["op"] == "route":
        how = dict(score=case["score"], renormalise=case["renormalise"], scale=case["scale"])
        w, experts = gs.route_experts(state["logits"], case["k"], bias=state["bias"], groups=case["groups"],
                                      groups_kept=case["kept"], group_score=case["group_score"], **how)
        out = {"weights": w, "experts": experts}
        if case["grad"]:
            out["d_logits"] = gs.route_experts_backward(state["d_weights"], state["logits"], experts, **how)
        return out
    if case["op"] == "logprobs":
        r = gs.token_logprobs(state["logits"], state["targets"], top=case["top"])
        out = {"logprobs": r.logprobs, "entropy": r.entropy}
        if case["top"]:
            out.update(top_logprobs=r.top_logprobs, top_ids=r.top_ids)
        if case["grad"]:
            out["d_logits"] = gs.token_logprobs_backward(state["d_logprobs"], state["d_entropy"], state["logits"], state["targets"], r)
        return out
    g = gs.group_by_expert(state["experts"], case["experts"], align=case["align"])
    if case["op"] == "group":
        return {"offsets": g.offsets, "counts": g.counts, "rows": g.rows, "positions": g.positions}
    out = {"rows": gs.dispatch_rows(state["x"], g), "out": gs.combine_rows(state["y"], g, state["weights"])}
    if case["grad"]:
        out["d_y"], out["d_weights"] = gs.combine_rows_backward(state["d_out"], state["y"], g, state["weights"])
        out["d_x"] = gs.combine_rows(state["d_rows"], g)
    return out


def run(state):
    return (_run_own if own else _run_plain)(state["case"], state)


# -------------------------------------------------------------------- work
def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "logprobs":
        values, rows = case["rows"] * case["vocab"], case["rows"]
        moved = values * size * (2 if case["grad"] else 1) + rows * (16 + 8 * case["top"] + (8 if case["grad"] else 0))
        return {"bytes": moved, "flops": values * (16 if case["grad"] else 8)}
    tokens, experts, pairs = case["tokens"], case["experts"], case["tokens"] * case["k"]
    if case["op"] == "route":
        moved = tokens * experts * size + pairs * 8 + (experts * 4 if case["bias"] else 0)
        if case["grad"]:
            moved += tokens * experts * size + pairs * 4
        return {"bytes": moved, "flops": tokens * experts * (12 if case["grad"] else 6)}
    capacity = _capacity(case)
    if case["op"] == "group":
        return {"bytes": 8 * pairs + 4 * capacity + 8 * experts, "flops": pairs}
    row = case["width"] * size
    moved = 4 * pairs + tokens * row + capacity * row      # experts, x, dispatched rows
    moved += 4 * pairs + pairs * row + tokens * row        # weights, expert outputs, combined rows
    flops = 2 * pairs * case["width"]
    if case["grad"]:
        moved += tokens * row + capacity * row + 4 * pairs + pairs * row + tokens * row  # d_out, d_y, d_weights, d_rows, d_x
        flops *= 3
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------- exact
def _exact_route(case, s):
    x = s["logits"].double()
    masked = torch.isneginf(x)
    if case["score"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(x, -1).nan_to_num(0.0)
    # the choice is by 32-bit numbers; scores that grow with the logits are compared as the logits
    c = s["logits"].float() if s["bias"] is None else p.float() + s["bias"]
    c = c.masked_fill(masked, -INF)
    groups, k = case["groups"], case["k"]
    if groups > 1:
        per = c.reshape(len(c), groups, -1)
        if case["group_score"] == "top2":
            per = per if s["bias"] is not None else p.float().masked_fill(masked, -INF).reshape(len(c), groups, -1)
            two = per.topk(2, -1).values
            value = two[..., 0] + two[..., 1].masked_fill(torch.isneginf(two[..., 1]), 0.0)
        else:
            value = per.max(-1).values
        order = value.argsort(dim=-1, descending=True, stable=True)
        place = order.argsort(dim=-1)
        c = c.reshape(len(c), groups, -1).masked_fill((place >= case["kept"]).unsqueeze(-1), -INF).reshape(c.shape)
    at = c.argsort(dim=-1, descending=True, stable=True)[:, :k]
    none = torch.isneginf(c.gather(1, at))
    chosen = torch.zeros_like(p).scatter(1, at, (~none).double())
    kept = p * chosen
    if case["renormalise"]:
        kept = (kept / kept.sum(-1, keepdim=True)).nan_to_num(0.0)
    out = {"weights": kept.gather(1, at) * case["scale"], "experts": None}
    if case["grad"]:
        g = torch.zeros_like(p).scatter(1, at, s["d_weights"].double().masked_fill(none, 0.0)) * case["scale"]
        if case["score"] == "softmax":  # renormalised: a softmax over the chosen ones
            q = kept if case["renormalise"] else p
            out["d_logits"] = q * (g - (g * q).sum(-1, keepdim=True))
        elif case["renormalise"]:
            mass = (p * chosen).sum(-1, keepdim=True)
            out["d_logits"] = (chosen * (g - (g * kept).sum(-1, keepdim=True)) / mass * p * (1 - p)).nan_to_num(0.0)
        else:
            out["d_logits"] = chosen * g * p * (1 - p)
    return out


def _exact_logprobs(case, s):
    logits, targets = s["logits"], s["targets"]
    parts = []
    for block in torch.arange(case["rows"], device=logits.device).split(1024):  # in 64 bits, some rows at a time
        x, t = logits[block].double(), targets[block]
        lse = torch.logsumexp(x, -1, keepdim=True)
        lp = x - lse
        lp[torch.isneginf(x)] = -INF
        p = lp.exp()
        h = -(p * lp.masked_fill(p == 0, 0.0)).sum(-1, keepdim=True)
        held = (t >= 0).unsqueeze(1)
        at = t.clamp(min=0).unsqueeze(1)
        part = [lp.gather(1, at).masked_fill(~held, 0.0).squeeze(1), h.squeeze(1)]
        if case["top"]:
            part.append(lp.topk(case["top"], -1).values)
        if case["grad"]:
            g = s["d_logprobs"][block].double().unsqueeze(1).masked_fill(~held, 0.0)
            u = s["d_entropy"][block].double().unsqueeze(1)
            dx = -p * (g + u * (lp.masked_fill(p == 0, 0.0) + h))
            alive = (~torch.isneginf(lse)).double()
            dx.scatter_add_(1, at, g * alive)
            part.append(dx)
        parts.append(part)
    whole = [torch.cat(v) for v in zip(*parts)]
    out = {"logprobs": whole[0], "entropy": whole[1]}
    if case["top"]:
        out.update(top_logprobs=whole[2], top_ids=None)
    if case["grad"]:
        out["d_logits"] = whole[-1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "logprobs":
        return _exact_logprobs(case, s)
    if case["op"] == "group":
        return None
    # every pair's place: groups in the experts' order, pairs of one expert in their own
    experts, k = s["experts"], case["k"]
    flat = experts.flatten().cpu().numpy()
    place, start, align = torch.full((flat.size,), -1, dtype=torch.int64), 0, case["align"]
    for e in range(case["experts"]):
        mine = torch.from_numpy((flat == e).nonzero()[0])
        place[mine] = start + torch.arange(len(mine))
        start += -(-len(mine) // align) * align
    place = place.to(experts.device)
    pair = (place >= 0).nonzero().squeeze(1)
    to, token = place[pair], pair // k
    rows = torch.zeros(_capacity(case), case["width"], dtype=s["x"].dtype, device=place.device)
    rows[to] = s["x"][token]
    w = s["weights"].flatten()[pair].double().unsqueeze(1)
    out = {"rows": rows}
    total = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device=place.device)
    out["out"] = total.index_add(0, token, s["y"][to].double() * w)
    if case["grad"]:
        d = s["d_out"][token].double()
        out["d_y"] = torch.zeros(rows.shape, dtype=torch.float64, device=place.device).index_copy(0, to, d * w)
        dw = torch.zeros(len(place), dtype=torch.float64, device=place.device)
        out["d_weights"] = dw.index_copy(0, pair, (d * s["y"][to].double()).sum(-1)).view(experts.shape)
        out["d_x"] = total.index_add(0, token, s["d_rows"][to].double())
    return out
