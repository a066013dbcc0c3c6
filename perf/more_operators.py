"""Cases of the operators around a language model's vocabulary and gradients: embedding lookup and its gradient, penalties,
biases and masks on logits, and the global norm of many gradients with clipping.

`run` computes them in plain torch operations, in 32 bits, or (own) with the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

INF = float("inf")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the last tokens of a few requests: only latency counts
        dict(name="embed decode", op="embed", tokens=8, vocab=32000, width=4096, dtype="bf16", scale=64.0, grad=False, padded=False),
        # a batch of long prompts
        dict(name="embed prefill", op="embed", tokens=16384, vocab=131072, width=4096, dtype="bf16", scale=1.0, grad=False, padded=False),
        # training steps: an odd table with padded tokens in 32 bits, and a large one whose frequent tokens come thousands of times
        dict(name="embed train odd", op="embed", tokens=8191, vocab=100003, width=1001, dtype="f32", scale=31.6, grad=True, padded=True),
        dict(name="embed train", op="embed", tokens=65536, vocab=131072, width=4096, dtype="bf16", scale=1.0, grad=True, padded=False),
        # answers: a few constrained requests, a serving batch with penalties, long histories on an odd vocabulary inside padded
        # rows, and a training step through the same adjustments
        dict(name="adjust decode", op="adjust", rows=4, vocab=32000, stride=32000, history=300, biases=16, allowed=True, dtype="bf16", grad=False),
        dict(name="adjust batch", op="adjust", rows=64, vocab=131072, stride=131072, history=2048, biases=0, allowed=False, dtype="f32", grad=False),
        dict(name="adjust long", op="adjust", rows=256, vocab=100003, stride=100096, history=16384, biases=300, allowed=True, dtype="bf16", grad=False),
        dict(name="adjust train", op="adjust", rows=2048, vocab=131072, stride=131072, history=1024, biases=64, allowed=True, dtype="bf16", grad=True),
        # gradients of a small model, of a middle one that the caches hold, of many odd tensors of two types, and of a large model
        dict(name="clip small", op="clip", tensors=12, elements=20011, dtype="f32", layout=1, clipped=True),
        dict(name="clip middle", op="clip", tensors=300, elements=1 << 24, dtype="f32", layout=2, clipped=True),
        dict(name="clip many", op="clip", tensors=1500, elements=(1 << 27) + 77, dtype="mixed", layout=3, clipped=True),
        dict(name="clip large", op="clip", tensors=200, elements=1 << 30, dtype="bf16", layout=4, clipped=True),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["embed", "adjust", "clip"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    size = 4 if dtype == "f32" else 2
    grad = rng.random() < 0.5
    if op == "embed":
        width = rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)])
        vocab = _log_int(rng, 1000, min(262144, (1 << 30) // (width * size)))
        return dict(op=op, tokens=_log_int(rng, 1, min(131072, (1 << 29) // (width * size))), vocab=vocab, width=width, dtype=dtype,
                    scale=rng.choice([1.0, round(width ** 0.5, 3)]), grad=grad, padded=rng.random() < 0.4)
    if op == "adjust":
        vocab = _log_int(rng, 1000, 200000)
        rows = _log_int(rng, 1, min(4096, (1 << 28) // vocab))
        history = 0 if rng.random() < 0.25 else _log_int(rng, 1, min(16384, (1 << 22) // rows))
        return dict(op=op, rows=rows, vocab=vocab, stride=vocab + rng.choice([0, 0, 1, 64]), history=history,
                    biases=rng.choice([0, 0, 1, 16, 300]), allowed=history == 0 or rng.random() < 0.5, dtype=dtype, grad=grad)
    elements = _log_int(rng, 1000, 1 << 28)
    return dict(op=op, tensors=_log_int(rng, 1, min(2000, elements // 8)), elements=elements, dtype=rng.choice([dtype, dtype, "mixed"]),
                layout=rng.randint(5, 1 << 20), clipped=rng.random() < 0.7)


def _sizes(case):
    """Elements of each tensor: some matrices hold most of them, many vectors the rest."""
    rng = random.Random(case["layout"])
    parts = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    share = (case["elements"] - case["tensors"]) / sum(parts)
    sizes = [1 + int(p * share) for p in parts]
    sizes[0] += case["elements"] - sum(sizes)
    return sizes


def _types(case):
    """The dtypes of a case's tensors: every third of a mixed one is kept in 32 bits."""
    if case["dtype"] != "mixed":
        return [case["dtype"]] * case["tensors"]
    return ["f32" if i % 3 == 0 else "bf16" for i in range(case["tensors"])]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def tokens_of(vocab, *shape):
        """Tokens of a text: the r-th most frequent one with a probability of about 1 / r."""
        rank = ((vocab + 1.0) ** uniform(*shape).double()).long().clamp(1, vocab) - 1
        return torch.randperm(vocab, generator=gen, device="cuda")[rank]

    state = {"case": case}
    if case["op"] == "embed":
        n, vocab, width, dtype = case["tokens"], case["vocab"], case["width"], DTYPES[case["dtype"]]
        state["table"] = torch.empty(vocab, width, dtype=dtype, device="cuda").normal_(0.0, 0.05, generator=gen)
        state["tokens"] = tokens_of(vocab, n)
        if case["padded"]:  # the ends of short sequences
            state["tokens"].masked_fill_(uniform(n) < 0.1, -1)
        if case["grad"]:
            state["d_out"] = torch.empty(n, width, dtype=dtype, device="cuda").normal_(generator=gen)
        return state

    if case["op"] == "adjust":
        rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        whole = torch.empty(rows, case["stride"], dtype=dtype, device="cuda")
        whole.normal_(0.0, 2.5, generator=gen)
        state["logits"] = whole[:, :vocab]
        for name in ("history", "prompt", "repetition", "presence", "frequency", "bias_tokens", "bias", "allowed"):
            state[name] = None
        if case["history"]:
            h = case["history"]
            lengths = (uniform(rows, 1) * h).long() + 1        # requests of different ages in one batch
            history = tokens_of(vocab, rows, h).masked_fill_(torch.arange(h, device="cuda") >= lengths, -1)
            state["history"] = history.to(torch.int32)
            state["prompt"] = (uniform(rows) * lengths.squeeze(1)).to(torch.int32)
            state["repetition"] = 1.0 + 0.1 * torch.randint(0, 4, (rows,), generator=gen, device="cuda")
            state["presence"] = 0.1 * torch.randint(0, 6, (rows,), generator=gen, device="cuda")
            state["frequency"] = 0.1 * torch.randint(0, 6, (rows,), generator=gen, device="cuda")
        if case["biases"]:      # no token twice
            first = torch.randint(vocab, (rows, 1), generator=gen, device="cuda")
            step = torch.arange(case["biases"], device="cuda") * (vocab // case["biases"])
            state["bias_tokens"] = ((first + step) % vocab).to(torch.int32)
            state["bias"] = normal(rows, case["biases"]) * 4.0
        if case["allowed"]:     # a third of the rows is free, in the others a grammar leaves a little or most of the vocabulary
            kind = torch.randint(3, (rows, 1), generator=gen, device="cuda")
            words = -(-vocab // 32)
            bits = torch.randint(-2 ** 31, 2 ** 31, (3, rows, words), generator=gen, device="cuda").to(torch.int32)
            little, most = bits[0] & bits[1] & bits[2], bits[0] | bits[1] | bits[2]
            state["allowed"] = torch.where(kind == 0, torch.full_like(little, -1), torch.where(kind == 1, little, most))
        if case["grad"]:
            state["d_out"] = torch.empty(rows, vocab, dtype=dtype, device="cuda").normal_(generator=gen)
        return state

    # the gradients of a type lie in one buffer, as its allocator would place them: at 512 bytes, or (odd layouts) one behind another
    sizes, types = _sizes(case), _types(case)
    state.update(flat={}, out={}, gradients=[], outs=[])
    room, at = {}, []
    for n, t in zip(sizes, types):
        at.append(room.get(t, 0))
        step = 1 if case["layout"] % 2 else 512 // (4 if t == "f32" else 2)
        room[t] = at[-1] + -(-n // step) * step
    for t, total in room.items():
        state["flat"][t] = torch.zeros(total, dtype=DTYPES[t], device="cuda")
        state["out"][t] = torch.zeros(total, dtype=DTYPES[t], device="cuda")
    for n, t, o in zip(sizes, types, at):
        g = state["flat"][t][o:o + n]
        g.normal_(0.0, 0.01, generator=gen)
        state["gradients"].append(g)
        state["outs"].append(state["out"][t][o:o + n])
    # some steps are clipped, others are not
    state["max_norm"] = 0.01 * case["elements"] ** 0.5 * (0.5 if seed % 3 else 2.0)
    return state


# ------------------------------------------------------------- plain forms
def _plain_embed(case, state):
    table, tokens, vocab = state["table"], state["tokens"], case["vocab"]
    held = ((tokens >= 0) & (tokens < vocab)).unsqueeze(1)
    at = torch.where(held.squeeze(1), tokens, 0)
    out = {"out": torch.where(held, table[at].float() * case["scale"], 0.0).to(table.dtype)}
    if case["grad"]:
        d = torch.where(held, state["d_out"].float(), 0.0)
        total = torch.zeros(vocab, case["width"], device=table.device).index_add_(0, at, d)
        out["d_table"] = total.mul_(case["scale"]).to(table.dtype)
    return out


def _plain_adjust(case, state):
    x, vocab = state["logits"].float(), case["vocab"]
    y, factor, allowed = x, None, None
    if state["history"] is not None:
        history = state["history"].long()
        held = (history >= 0) & (history < vocab)
        at = torch.where(held, history, 0)
        mine = held & (torch.arange(history.shape[1], device=x.device) >= state["prompt"].unsqueeze(1))
        count = torch.zeros_like(x).scatter_add_(1, at, mine.float())
        seen = torch.zeros_like(x).scatter_add_(1, at, held.float()) > 0
        r = state["repetition"].unsqueeze(1)
        y = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        y = y - (state["frequency"].unsqueeze(1) * count + state["presence"].unsqueeze(1) * (count > 0))
        factor = torch.where(seen, torch.where(x > 0, 1.0 / r, r), 1.0)
    if state["bias"] is not None:
        y = y + torch.zeros_like(x).scatter_(1, state["bias_tokens"].long(), state["bias"])
    if state["allowed"] is not None:
        bit = torch.arange(32, dtype=torch.int32, device=x.device)
        allowed = (((state["allowed"].unsqueeze(2) >> bit) & 1) > 0).view(case["rows"], -1)[:, :vocab]
        y = torch.where(allowed, y, -INF)
    out = {"logits": y.to(state["logits"].dtype)}
    if case["grad"]:
        d = state["d_out"].float()
        d = d if factor is None else d * factor
        d = d if allowed is None else torch.where(allowed, d, 0.0)
        out["d_logits"] = d.to(state["logits"].dtype)
    return out


def _plain_clip(case, state):
    # between the tensors the buffers hold zeros
    squares = [g.float().square().sum(dtype=torch.float64) for g in state["flat"].values()]
    norm = torch.stack(squares).sum().sqrt()
    out = {"norm": norm.float()}
    if case["clipped"]:
        c = torch.where(norm > state["max_norm"], state["max_norm"] / norm, 1.0).float()
        out["gradients"] = {t: (g.float() * c).to(g.dtype) for t, g in state["flat"].items()}
    return out


# --------------------------------------------------------------------- run
def _run_own(case, state):
    import bitonic_networks_gb300 as gs
    if case["op"] == "embed":
        out = {"out": gs.embed_tokens(state["table"], state["tokens"], scale=case["scale"])}
        if case["grad"]:
            out["d_table"] = gs.embed_tokens_backward(state["d_out"], state["tokens"], case["vocab"], scale=case["scale"])
        return out
    if case["op"] == "adjust":
        how = {k: state[k] for k in ("history", "repetition", "allowed")}
        out = {"logits": gs.adjust_logits(state["logits"], prompt=state["prompt"], presence=state["presence"], frequency=state["frequency"],
                                          bias_tokens=state["bias_tokens"], bias=state["bias"], **how)}
        if case["grad"]:
            out["d_logits"] = gs.adjust_logits_backward(state["d_out"], state["logits"], **how)
        return out
    if case["clipped"]:
        return {"norm": gs.clip_gradients(state["gradients"], state["max_norm"], out=state["outs"]).norm, "gradients": state["out"]}
    return {"norm": gs.gradient_norm(state["gradients"])}


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"embed": _plain_embed, "adjust": _plain_adjust, "clip": _plain_clip}[case["op"]](case, state)


# -------------------------------------------------------------------- work
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "embed":
        n, vocab, row = case["tokens"], case["vocab"], case["width"] * size
        r = np.arange(1, vocab + 1, dtype=np.float64)
        p = np.log1p(1.0 / r) / math.log(vocab + 1.0)
        different = float((1.0 - (1.0 - p) ** n).sum())        # tokens that come up, on average
        moved, flops = 8 * n + (different + n) * row, n * case["width"]
        if case["grad"]:
            moved, flops = moved + (n + vocab) * row, 3 * flops
        return {"bytes": int(moved), "flops": flops}
    if case["op"] == "adjust":
        values, rows, words = case["rows"] * case["vocab"], case["rows"], -(-case["vocab"] // 32)
        moved = 2 * values * size + rows * (4 * case["history"] + 8 * case["biases"] + (4 * words if case["allowed"] else 0) + 16)
        if case["grad"]:
            moved += 2 * values * size
        return {"bytes": moved, "flops": (2 if case["grad"] else 1) * values + 4 * rows * case["history"]}
    moved = sum(n * (4 if t == "f32" else 2) for n, t in zip(_sizes(case), _types(case)))
    return {"bytes": moved * (2 if case["clipped"] else 1) + 4, "flops": case["elements"] * (3 if case["clipped"] else 2)}


# ------------------------------------------------------------------- exact
def _exact_embed(case, s):
    inside = ((s["tokens"] >= 0) & (s["tokens"] < case["vocab"])).nonzero().squeeze(1)
    token = s["tokens"][inside]
    out = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device=token.device)
    out[inside] = s["table"][token].double() * case["scale"]
    result = {"out": out}
    if case["grad"]:
        # a token's rows one behind another, summed a block of the table's columns at a time
        token, order = torch.sort(token, stable=True)
        d_table = torch.zeros(case["vocab"], case["width"], dtype=torch.float64, device=token.device)
        for c in range(0, case["width"], 512):
            d = s["d_out"][inside[order], c:c + 512].double()
            d_table[:, c:c + 512].index_add_(0, token, d * case["scale"])
        result["d_table"] = d_table
    return result


def _exact_adjust(case, s):
    x, vocab = s["logits"].double(), case["vocab"]
    dx = s["d_out"].double() if case["grad"] else None
    shift = torch.arange(vocab, device=x.device) % 32
    for i in range(case["rows"]):
        row = x[i]
        if s["history"] is not None:
            told = s["history"][i].long()
            own_part = told[int(s["prompt"][i]):]
            ever = torch.unique(told[(told >= 0) & (told < vocab)])
            r, old = float(s["repetition"][i]), row[ever].clone()
            by = torch.where(old > 0, torch.full_like(old, 1.0 / r), torch.full_like(old, r))
            row[ever] = old * by
            if dx is not None:
                dx[i, ever] *= by
            new, times = torch.unique(own_part[(own_part >= 0) & (own_part < vocab)], return_counts=True)
            row[new] -= float(s["frequency"][i]) * times.double() + float(s["presence"][i])
        if s["bias"] is not None:
            row[s["bias_tokens"][i].long()] += s["bias"][i].double()
        if s["allowed"] is not None:
            word = s["allowed"][i].long().repeat_interleave(32)[:vocab]
            no = (word.bitwise_right_shift(shift) & 1) == 0
            row[no] = -INF
            if dx is not None:
                dx[i, no] = 0.0
    return {"logits": x, "d_logits": dx} if case["grad"] else {"logits": x}


def _exact_clip(case, s):
    square = 0.0
    for g in s["gradients"]:
        square += sum(float((part.double() ** 2).sum()) for part in g.split(1 << 26))
    norm = math.sqrt(square)
    out = {"norm": torch.tensor(norm, dtype=torch.float64)}
    if case["clipped"]:
        by = min(1.0, s["max_norm"] / norm)
        out["gradients"] = {t: g.double().mul_(by) for t, g in s["flat"].items()}
    return out


def exact(case, seed):
    return {"embed": _exact_embed, "adjust": _exact_adjust, "clip": _exact_clip}[case["op"]](case, prepare(case, seed))
