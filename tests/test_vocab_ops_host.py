"""Host-side checks of embedding, adjusted logits and gradient norm that need no GPU:
workspace sizes, and argument errors found before the device is touched."""
import ctypes

import pytest

A, B, C, D, E, W = (0x10000000 * (i + 1) for i in range(6))      # no memory behind them
OK, EINVAL, EALIGN, EWS, ETOOBIG = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from bitonic_networks_gb300 import _lib
    return _lib.load()


def test_package_exports():
    import bitonic_networks_gb300 as gs
    for name in ("embed_tokens", "embed_tokens_backward", "embed_workspace_bytes", "adjust_logits", "adjust_logits_backward", "gradient_norm",
                 "clip_gradients", "ClippedGradients"):
        assert callable(getattr(gs, name)) and name in gs.__all__


def test_workspace_sizes(lib):
    ws = lib.gsort_embed_tokens_backward_workspace_bytes
    assert ws(0, 9, 64, 0) == ws(-1, 9, 64, 0) == ws(1 << 30, 9, 64, 0) == ws(5, 9, 0, 0) == ws(5, 9, 64, 3) == ws(5, 9, 1 << 30, 0) == 0
    assert ws(5, 0, 64, 0) == ws(5, 1 << 30, 64, 0) == 0
    for n in (1, 8192, 8193, 1 << 20, (1 << 30) - 1):
        for width, dtype in ((1, 1), (64, 0), (1001, 2), (8192, 1)):
            assert ws(n, 9, width, dtype) >= 8 * n and ws(n, 9, width, dtype) % 256 == 0
    # the partial sums take an eighth of what the gradient itself takes, at most, where it is large
    assert ws(65536, 131072, 4096, 1) < 65536 * 4096 * 2 / 8 + 65536 * 64 + (8 << 20)
    norm = lib.gsort_gradient_norm_workspace_bytes
    assert norm(0) == norm(-1) == norm(1 << 30) == 0 and 0 < norm(1) == norm(1000) < norm(1001) == norm(2000)


def test_embed_argument_errors(lib):
    def call(table=A, dtype=0, vocab=10, width=8, stride=8, tokens=B, tb=8, n=4, scale=1.0, out=C):
        return lib.gsort_embed_tokens(table, dtype, vocab, width, stride, tokens, tb, n, scale, out, None)

    assert call(n=0, table=None, tokens=None, out=None) == OK
    for bad in (dict(dtype=3), dict(vocab=0), dict(width=0, stride=0), dict(stride=7), dict(stride=0), dict(tb=2), dict(n=-1), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(table=None), dict(tokens=None), dict(out=None), dict(out=A + 32), dict(out=B)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(vocab=1 << 30), dict(n=1 << 30), dict(width=1 << 30, stride=1 << 30)):
        assert call(**bad) == ETOOBIG, bad
    for bad in (dict(table=A + 2), dict(out=C + 1), dict(tokens=B + 4), dict(dtype=1, table=A + 1)):
        assert call(**bad) == EALIGN, bad

    def back(d=A, dtype=0, n=4, width=8, stride=8, tokens=B, tb=4, vocab=10, scale=1.0, acc=0, out=C, ostride=8, ws=W, nbytes=1 << 30):
        return lib.gsort_embed_tokens_backward(d, dtype, n, width, stride, tokens, tb, vocab, scale, acc, out, ostride, ws, nbytes, None)

    assert back(n=0, acc=1, d=None, tokens=None) == OK
    for bad in (dict(dtype=-1), dict(vocab=0), dict(stride=7), dict(ostride=7), dict(tb=1), dict(n=-1), dict(scale=float("nan")), dict(d=None),
                dict(tokens=None), dict(out=None), dict(out=A), dict(out=B), dict(ws=A, nbytes=1 << 12), dict(ws=C)):
        assert back(**bad) == EINVAL, bad
    assert back(vocab=1 << 30) == ETOOBIG and back(n=1 << 30) == ETOOBIG
    assert back(ws=None) == EWS and back(nbytes=16) == EWS and back(ws=W + 8) == EALIGN
    assert back(d=A + 2) == EALIGN and back(out=C + 2) == EALIGN and back(tokens=B + 2) == EALIGN


def test_adjust_argument_errors(lib):
    from bitonic_networks_gb300 import _lib

    def how(**fields):
        full = dict(d_history=B, length=6, history_stride=6, history_bytes=4, d_prompt=B + 0x1000, d_repetition=B + 0x2000, d_presence=None,
                    d_frequency=None, d_bias_tokens=B + 0x3000, d_bias=B + 0x4000, biases=3, bias_stride=3, bias_bytes=8, d_allowed=B + 0x5000,
                    allowed_stride=4)
        return _lib.Adjustments(**{**full, **fields})

    def call(x=A, dtype=0, rows=4, vocab=100, stride=100, out=C, ostride=100, **fields):
        return lib.gsort_adjust_logits(x, dtype, rows, vocab, stride, how(**fields), out, ostride, None)

    assert call(rows=0, x=None, out=None) == OK
    for bad in (dict(dtype=4), dict(rows=-1), dict(vocab=0, stride=0, ostride=0), dict(stride=99), dict(ostride=99), dict(x=None), dict(out=None),
                dict(length=-1), dict(biases=-1), dict(history_bytes=2), dict(history_stride=5), dict(d_history=None), dict(d_bias=None),
                dict(d_bias_tokens=None), dict(bias_bytes=1), dict(bias_stride=2), dict(allowed_stride=3), dict(out=A + 16), dict(out=A, ostride=101),
                dict(out=B), dict(out=B + 0x5000)):
        assert call(**bad) == EINVAL, bad
    assert lib.gsort_adjust_logits(A, 0, 4, 100, 100, None, C, 100, None) == EINVAL
    for bad in (dict(rows=1 << 30), dict(vocab=1 << 30, stride=1 << 30, ostride=1 << 30)):
        assert call(**bad) == ETOOBIG, bad
    for bad in (dict(x=A + 2), dict(out=C + 2), dict(d_history=B + 2), dict(d_prompt=B + 0x1001), dict(d_repetition=B + 0x2002),
                dict(d_bias_tokens=B + 0x3004), dict(d_bias=B + 0x4002), dict(d_allowed=B + 0x5001)):
        assert call(**bad) == EALIGN, bad

    def back(d=A, rows=4, stride=100, x=D, xstride=100, out=C, ostride=100, **fields):
        return lib.gsort_adjust_logits_backward(d, 1, rows, 100, stride, x, xstride, how(**fields), out, ostride, None)

    assert back(rows=0) == OK
    for bad in (dict(d=None), dict(x=None), dict(xstride=99), dict(out=None), dict(out=D), dict(out=A, ostride=101), dict(out=B)):
        assert back(**bad) == EINVAL, bad
    assert back(x=D + 1) == EALIGN and back(out=C + 1) == EALIGN


def test_norm_argument_errors(lib):
    def lists(ins, outs, sizes, dtypes):
        n = len(sizes)
        return ((ctypes.c_void_p * n)(*ins), (ctypes.c_void_p * n)(*outs) if outs is not None else None, (ctypes.c_int64 * n)(*sizes),
                (ctypes.c_int * n)(*dtypes))

    def norm(ins=(A, B), sizes=(10, 20), dtypes=(0, 1), count=2, out=C, ws=W, nbytes=1 << 20):
        i, _, s, t = lists(ins, None, sizes, dtypes)
        return lib.gsort_gradient_norm(i, s, t, count, out, ws, nbytes, None)

    for bad in (dict(count=-1), dict(out=None), dict(sizes=(10, -1)), dict(dtypes=(0, 3)), dict(ins=(A, None)), dict(out=A + 8), dict(ws=A)):
        assert norm(**bad) == EINVAL, bad
    assert lib.gsort_gradient_norm(None, None, None, 2, C, W, 1 << 20, None) == EINVAL
    assert norm(sizes=(10, 1 << 50)) == ETOOBIG
    assert norm(ws=None) == EWS and norm(nbytes=8) == EWS and norm(ws=W + 8) == EALIGN and norm(ins=(A + 2, B)) == EALIGN and norm(out=C + 2) == EALIGN

    def clip(ins=(A, B), outs=(C, D), sizes=(10, 20), dtypes=(0, 0), limit=1.0, scale=1.0, norm=E, ws=W):
        i, o, s, t = lists(ins, outs, sizes, dtypes)
        return lib.gsort_clip_gradients(i, o, s, t, len(sizes), limit, scale, norm, ws, 1 << 20, None)

    for bad in (dict(limit=-1.0), dict(limit=float("nan")), dict(scale=float("inf")), dict(outs=(C, None)), dict(outs=None), dict(outs=(C, C)),
                dict(outs=(C, C + 36)), dict(outs=(B, A)), dict(outs=(A + 4, D)), dict(outs=(C, A + 36)), dict(norm=C), dict(norm=A + 4),
                dict(ins=(A, A), outs=(A, A)), dict(ins=(A, A), outs=(A, D)), dict(ws=C)):
        assert clip(**bad) == EINVAL, bad
    assert clip(outs=(C + 1, D)) == EALIGN


def test_torch_wrappers_refuse_before_the_device():
    import torch

    import bitonic_networks_gb300 as gs
    x, t = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: gs.embed_tokens(x, t), lambda: gs.embed_tokens_backward(x, t, 9), lambda: gs.adjust_logits(x),
                 lambda: gs.adjust_logits_backward(x, x), lambda: gs.gradient_norm([x]), lambda: gs.clip_gradients([x], 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: gs.embed_tokens(x.double(), t), lambda: gs.adjust_logits(x.int()), lambda: gs.gradient_norm([1.0]), lambda: gs.gradient_norm(1.0),
                 lambda: gs.clip_gradients([x.long()], 1.0)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        gs.gradient_norm([])
    with pytest.raises(RuntimeError):
        gs.adjust_logits(x, history=t.view(4, 1).int(), repetition=torch.ones(4, requires_grad=True))


def test_outputs_that_require_a_gradient_are_refused():
    """Nothing of these calls is recorded: an output that is in a graph would go on with its old gradient."""
    import torch

    import bitonic_networks_gb300 as gs
    x, t = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    leaf = torch.zeros(4, 64, requires_grad=True)
    for out in (leaf, leaf * 1.0, (leaf * 1.0)[:]):
        for call in (lambda: gs.adjust_logits(x, out=out), lambda: gs.adjust_logits(out.detach(), out=out),
                     lambda: gs.adjust_logits_backward(x, None, out=out), lambda: gs.embed_tokens_backward(x, t, 4, out=out),
                     lambda: gs.embed_tokens_backward(x, t, 4, out=out, accumulate=True)):
            with pytest.raises(RuntimeError, match="no gradient"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call()


def test_options_of_extended_calls(lib):
    """What the options may hold is checked before anything else; NULL options are the defaults."""
    from bitonic_networks_gb300 import _lib
    bad = [_lib.Options(0, -1, None, 0, 1), _lib.Options(0, -1, None, -1, 0), _lib.Options(0, -1, None, 2, 0)]
    i, s, t = (ctypes.c_void_p * 1)(A), (ctypes.c_int64 * 1)(10), (ctypes.c_int * 1)(0)
    how = _lib.Adjustments()
    for o in bad:
        assert lib.gsort_gradient_norm_ex(i, s, t, 1, C, W, 1 << 20, None, ctypes.byref(o)) == EINVAL
        assert lib.gsort_clip_gradients_ex(i, i, s, t, 1, 1.0, 1.0, C, W, 1 << 20, None, ctypes.byref(o)) == EINVAL
        assert lib.gsort_adjust_logits_ex(A, 0, 4, 100, 100, how, C, 100, None, ctypes.byref(o)) == EINVAL
        assert lib.gsort_embed_tokens_backward_ex(A, 0, 4, 8, 8, B, 4, 10, 1.0, 0, C, 8, W, 1 << 30, None, ctypes.byref(o)) == EINVAL
        assert lib.gsort_adjust_logits_backward_ex(A, 0, 4, 100, 100, None, 0, how, C, 100, None, ctypes.byref(o)) == EINVAL
    assert lib.gsort_gradient_norm_ex(i, s, t, 1, C, W, 8, None, None) == EWS
    assert lib.gsort_clip_gradients_ex(i, i, s, t, 1, 1.0, 1.0, C, W, 8, None, None) == EWS
    assert lib.gsort_clip_gradients_ex(i, None, s, t, 1, 1.0, 1.0, C, W, 1 << 20, None, None) == EINVAL
    assert lib.gsort_adjust_logits_ex(A, 0, 4, 100, 99, how, C, 100, None, None) == EINVAL
    assert lib.gsort_adjust_logits_ex(None, 0, 0, 100, 100, how, None, 100, None, None) == OK
    assert lib.gsort_embed_tokens_backward_ex(A, 0, 4, 8, 8, B, 4, 10, 1.0, 0, C, 8, W, 16, None, None) == EWS
    assert lib.gsort_embed_tokens_backward_ex(None, 0, 0, 8, 8, None, 4, 10, 1.0, 1, C, 8, None, 0, None, None) == OK
    assert lib.gsort_adjust_logits_backward_ex(None, 0, 0, 100, 100, None, 0, how, None, 100, None, None) == OK
