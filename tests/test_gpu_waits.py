"""Waits of the operators around the vocabulary and the gradients that run out: a testing option
makes the waits of one CTA (of the sort: one tile) give up at once.  The kernels end, the result says
that something is missing, other rows and the next call are right."""
import ctypes
import math

import pytest
import torch

import bitonic_networks_gb300 as gs
from bitonic_networks_gb300 import _lib
from model_ref import DTYPES

pytestmark = pytest.mark.gpu
OK, ETIMEOUT = 0, -6
CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def options(**fields):
    return ctypes.byref(_lib.Options(fields.get("spin_limit", 0), fields.get("stall_tile", -1), None, 0, 0))


def stream():
    return torch.cuda.current_stream().cuda_stream


def lists(tensors):
    n = len(tensors)
    return ((ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]), (ctypes.c_int64 * n)(*[t.numel() for t in tensors]),
            (ctypes.c_int * n)(*[CODES[t.dtype] for t in tensors]))


def norm_space(count):
    return torch.empty(_lib.load().gsort_gradient_norm_workspace_bytes(count), dtype=torch.uint8, device="cuda")


def norm(tensors, **fields):
    at, sizes, codes = lists(tensors)
    out, ws = torch.full((), 7.0, device="cuda"), norm_space(len(tensors))
    assert _lib.load().gsort_gradient_norm_ex(at, sizes, codes, len(tensors), out.data_ptr(), ws.data_ptr(), ws.numel(), stream(),
                                              options(**fields)) == OK
    return float(out)


# CTAs with several steps each, some with one; more tensors than one launch takes
GRADIENTS = {"many steps": [30_000_001, 77, 5_000_000], "one step": [5000, 4096, 3], "two launches": [9000] * 1300}


@pytest.mark.parametrize("name", GRADIENTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_norm_without_all_of_its_parts_is_nan(name, dtype):
    tensors = [torch.randn(n, device="cuda").to(dtype) for n in GRADIENTS[name]]
    want = float(gs.gradient_norm(tensors))
    for stall in (0, 1):
        assert math.isnan(norm(tensors, stall_tile=stall, spin_limit=100)), stall
        assert float(gs.gradient_norm(tensors)) == want
    assert norm(tensors) == want == norm(tensors, stall_tile=10 ** 6) == norm(tensors, spin_limit=1 << 22)


def test_a_norm_without_copies_waits_for_nothing():
    tensors = [torch.ones(3, device="cuda"), torch.ones(1, dtype=torch.bfloat16, device="cuda")]
    assert norm(tensors, stall_tile=0) == 2.0


def clip(tensors, out, max_norm, **fields):
    at, sizes, codes = lists(tensors)
    got, ws = torch.full((), 7.0, device="cuda"), norm_space(len(tensors))
    assert _lib.load().gsort_clip_gradients_ex(at, lists(out)[0], sizes, codes, len(tensors), max_norm, 1.0, got.data_ptr(), ws.data_ptr(),
                                               ws.numel(), stream(), options(**fields)) == OK
    return float(got)


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


@pytest.mark.parametrize("name", GRADIENTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("off", [0, 1])
def test_gradients_that_did_not_come_are_nan(name, dtype, off):
    """Every result is what it should be or NaN, none is left as it was, and the norm tells of it."""
    tensors = [torch.randn(n, device="cuda").to(dtype) for n in GRADIENTS[name]]
    limit = 0.5 * float(gs.gradient_norm(tensors))
    want = gs.clip_gradients(tensors, limit)
    for stall in (0, 1):
        for in_place in (False, True):
            out = [t.clone() if in_place else torch.full((t.numel() + off,), 9.0, dtype=dtype, device="cuda")[off:] for t in tensors]
            got = clip(out if in_place else tensors, out, limit, stall_tile=stall, spin_limit=100)
            assert math.isnan(got), (stall, in_place)
            lost = [int(t.isnan().sum()) for t in out]
            assert all(bool((t.isnan() | (bits(t) == bits(w))).all()) for t, w in zip(out, want.gradients))
            assert sum(lost) >= 4 and (name != "two launches" or (sum(lost[:1000]) > 0 and sum(lost[1000:]) > 0))
            assert sum(lost) % (16 // out[0].element_size()) == 0          # whole vectors: tensors' ends come by themselves
            assert sum(lost) < sum(t.numel() for t in out)
    again = [torch.empty_like(t) for t in tensors]
    for fields in ({}, dict(stall_tile=10 ** 6), dict(spin_limit=1 << 22)):
        assert clip(tensors, again, limit, **fields) == float(want.norm)
        assert all(torch.equal(bits(a), bits(w)) for a, w in zip(again, want.gradients))


def test_gradients_that_stay_as_they_are_need_not_come():
    tensors = [torch.randn(100_000, device="cuda"), torch.randn(33, device="cuda")]
    before = [t.clone() for t in tensors]
    assert math.isnan(clip(tensors, tensors, 1e9, stall_tile=0))
    assert all(torch.equal(a, b) for a, b in zip(tensors, before))


def adjust(x, how, allowed, out, d=None, **fields):
    h = how["history"]
    a = _lib.Adjustments(d_history=h.data_ptr(), length=h.shape[1], history_stride=h.shape[1], history_bytes=h.element_size(),
                         d_repetition=how["repetition"].data_ptr(), d_bias_tokens=how["bias_tokens"].data_ptr(), d_bias=how["bias"].data_ptr(),
                         biases=how["bias"].shape[1], bias_stride=how["bias"].shape[1], bias_bytes=how["bias_tokens"].element_size(),
                         d_allowed=allowed.data_ptr(), allowed_stride=allowed.shape[1])
    rows, vocab = x.shape
    if d is None:
        rc = _lib.load().gsort_adjust_logits_ex(x.data_ptr(), CODES[x.dtype], rows, vocab, vocab, ctypes.byref(a), out.data_ptr(), vocab, stream(),
                                                options(**fields))
    else:
        rc = _lib.load().gsort_adjust_logits_backward_ex(d.data_ptr(), CODES[x.dtype], rows, vocab, vocab, x.data_ptr(), vocab, ctypes.byref(a),
                                                         out.data_ptr(), vocab, stream(), options(**fields))
    assert rc == OK
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,length,whole", [(3, 60011, 40, False), (400, 9001, 300, True), (200, 40000, 9000, True), (310, 300000, 50, True)])
@pytest.mark.parametrize("backward", [False, True])
def test_logits_that_did_not_come_are_nan(dtype, rows, vocab, length, whole, backward):
    """Other rows are right, and so is what is read by itself; `whole`: a row is one CTA's."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, d = (torch.randn(rows, vocab, generator=g, device="cuda").to(dtype) for _ in range(2))
    how = dict(history=torch.randint(vocab, (rows, length), generator=g, device="cuda"), repetition=torch.rand(rows, generator=g, device="cuda") + 0.5,
               bias_tokens=torch.randint(vocab, (rows, 7), generator=g, device="cuda"), bias=torch.randn(rows, 7, generator=g, device="cuda"))
    allowed = torch.full((rows, (vocab + 31) // 32), -1, dtype=torch.int32, device="cuda")
    grad = d if backward else None
    want = gs.adjust_logits_backward(d, x, history=how["history"], repetition=how["repetition"], allowed=allowed) if backward else \
        gs.adjust_logits(x, **how, allowed=allowed)
    for stall in (0, 7):
        got = adjust(x, how, allowed, torch.full_like(x, 9.0), grad, stall_tile=stall, spin_limit=100)
        lost = got.isnan().sum(1)
        assert int((lost > 0).sum()) == 1 and (not whole or vocab == 300000 or int(lost[stall]) > 0), lost
        row = int(lost.argmax())
        assert bool((got.isnan() | (bits(got) == bits(want))).all())
        named = how["history"][row] if backward else torch.cat([how["history"][row], how["bias_tokens"][row]])
        assert not bool(got[row, named].isnan().any())
        if whole and vocab < 300000:            # all but those and the row's cut ends
            others = torch.ones(vocab, dtype=torch.bool, device="cuda")
            others[named] = False
            vector = 16 // x.element_size()
            assert int(lost[row]) >= int(others.sum()) - 2 * (vector - 1)
    for fields in ({}, dict(stall_tile=10 ** 6), dict(spin_limit=1 << 22)):
        assert torch.equal(bits(adjust(x, how, allowed, torch.full_like(x, 9.0), grad, **fields)), bits(want))
    into = (d if backward else x).clone()
    assert torch.equal(bits(adjust(x if backward else into, how, allowed, into, into if backward else None, stall_tile=0)), bits(want))     # in place nothing is copied


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,width", [(30000, 5000, 40), (70001, 900, 33), (300001, 70000, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_sort_of_tokens_that_gives_up(dtype, n, vocab, width, accumulate):
    """Rows of tokens that occur are NaN, others zero or as they were, and the workspace tells of it.  One cooperative kernel
    sorts up to 2^18 tokens here, passes with look-backs more."""
    lib, g = _lib.load(), torch.Generator(device="cuda").manual_seed(n)
    tokens = torch.randint(vocab, (n,), generator=g, device="cuda") // 3 * 3         # a third of the rows
    tokens[:50] = -1
    tokens[50:60] = vocab
    d, old = torch.randn(n, width, generator=g, device="cuda").to(dtype), torch.randn(vocab, width + 3, generator=g, device="cuda").to(dtype)
    ws = torch.empty(gs.embed_workspace_bytes(n, vocab, width, dtype), dtype=torch.uint8, device="cuda")
    held = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    held[tokens[60:]] = True

    def call(**fields):
        out = old.clone()
        rc = lib.gsort_embed_tokens_backward_ex(d.data_ptr(), CODES[dtype], n, width, width, tokens.data_ptr(), 8, vocab, 1.0, int(accumulate),
                                                out.data_ptr(), width + 3, ws.data_ptr(), ws.numel(), stream(), options(**fields))
        assert rc == OK
        return out, lib.gsort_check(ws.data_ptr(), stream())

    want, status = call()
    assert status == OK and not bool(want.isnan().any())
    for stall in (0, 1):
        got, status = call(stall_tile=stall, spin_limit=2000)
        assert status == ETIMEOUT
        assert bool(got[held, :width].isnan().all())
        assert torch.equal(bits(got[~held].contiguous()), bits(want[~held].contiguous())) and torch.equal(got[:, width:], old[:, width:])
        if accumulate:
            assert torch.equal(got[~held], old[~held])
        again, status = call()
        assert status == OK and torch.equal(bits(again), bits(want))
