"""Host-side checks of the language-model operators that need no GPU: sizes, and
argument errors found before the device is touched."""
import pytest

A, B, C, D, W = 0x10000000, 0x20000000, 0x30000000, 0x50000000, 0x40000000   # no memory behind them
OK, EINVAL, EALIGN, EWS, ETOOBIG = 0, -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from bitonic_networks_gb300 import _lib
    return _lib.load()


def test_package_exports():
    import bitonic_networks_gb300 as gs
    for name in ("route_experts", "group_by_expert", "dispatch_rows", "combine_rows", "token_logprobs",
                 "token_logprobs_backward", "sort_pairs"):
        assert callable(getattr(gs, name))


def test_group_sizes(lib):
    cap, ws = lib.gsort_group_capacity, lib.gsort_group_workspace_bytes
    for pairs, experts, align in ((1, 1, 1), (7, 256, 16), (4096, 8, 128), (100_003, 60, 7), ((1 << 30) - 1, 1024, 1)):
        most = pairs + min(pairs, experts) * (align - 1)
        assert cap(pairs, experts, align) == most // align * align >= pairs
    assert cap(0, 8, 128) == 0 and cap(-1, 8, 1) == 0 and cap(8, 0, 1) == 0 and cap(8, 1025, 1) == 0 and cap(8, 8, 0) == 0
    assert cap((1 << 30) - 1, 1024, 128) == 0            # above the largest layout
    assert ws(4096, 1024) == 0 and ws(4097, 60) == 2 * 60 * 4
    assert ws(1 << 29, 60) == 148 * 60 * 4 and ws(-1, 8) == 0 and ws(8, 1025) == 0


def test_route_argument_errors(lib):
    f = lib.gsort_route_experts

    def call(x=A, dtype=0, tokens=4, experts=16, stride=16, bias=None, score=0, groups=1, kept=1, how=0, k=2, scale=1.0, w=B, e=C):
        return f(x, dtype, tokens, experts, stride, bias, score, groups, kept, how, k, 0, scale, w, e, None)

    assert call(tokens=0, x=None, w=None, e=None) == OK
    for bad in (dict(dtype=3), dict(dtype=-1), dict(tokens=-1), dict(experts=0), dict(stride=15), dict(score=2), dict(groups=0),
                dict(groups=3), dict(groups=33, experts=33, stride=33), dict(groups=4, kept=5), dict(groups=4, kept=0), dict(how=2),
                dict(k=0), dict(k=17), dict(scale=float("inf")), dict(scale=float("nan")), dict(x=None), dict(w=None), dict(e=None),
                dict(w=A + 4), dict(e=B + 16), dict(bias=B)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(experts=1025, stride=1025), dict(tokens=1 << 30), dict(k=33, experts=64, stride=64)):
        assert call(**bad) == ETOOBIG, bad
    for bad in (dict(x=A + 2), dict(dtype=1, x=A + 1), dict(w=B + 2), dict(e=C + 1), dict(bias=D + 2)):
        assert call(**bad) == EALIGN, bad
    g = lib.gsort_route_experts_backward
    assert g(A, B, 0, 0, 16, 16, C, 2, 0, 0, 1.0, D, None) == OK
    assert g(A, B, 0, 4, 16, 16, C, 2, 0, 0, 1.0, B, None) == EINVAL       # the gradient over the logits
    assert g(None, B, 0, 4, 16, 16, C, 2, 0, 0, 1.0, D, None) == EINVAL
    assert g(A, B, 0, 4, 16, 16, C, 2, 0, 0, 1.0, D + 2, None) == EALIGN
    assert g(A, B, 0, 4, 16, 16, C, 2, 9, 0, 1.0, D, None) == EINVAL


def test_group_argument_errors(lib):
    def call(e=A, pairs=10, experts=4, align=1, off=B, cnt=B + 0x1000, rows=C, cap=10, pos=D, ws=None, nbytes=0):
        return lib.gsort_group_by_expert(e, pairs, experts, align, off, cnt, rows, cap, pos, ws, nbytes, None)

    for bad in (dict(pairs=-1), dict(experts=0), dict(align=0), dict(cap=9), dict(cap=-1), dict(e=None), dict(off=None), dict(cnt=None),
                dict(rows=None), dict(pos=None), dict(cnt=B + 16), dict(pos=A), dict(rows=D + 4)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(pairs=1 << 30, cap=1 << 30), dict(experts=1025), dict(experts=1024, pairs=1 << 20, align=1 << 30)):
        assert call(**bad) == ETOOBIG, bad
    for bad in (dict(e=A + 2), dict(off=B + 1), dict(pos=D + 3)):
        assert call(**bad) == EALIGN, bad
    assert call(pairs=5000, cap=5000) == EWS
    assert call(pairs=5000, cap=5000, ws=W, nbytes=8) == EWS
    assert call(pairs=5000, cap=5000, ws=W + 8, nbytes=1 << 20) == EALIGN
    assert call(pairs=5000, cap=5000, ws=A, nbytes=1 << 20) == EINVAL      # over the experts


def test_rows_argument_errors(lib):
    def dispatch(x=A, dtype=0, tokens=4, width=8, stride=8, pos=B, k=2, rows=B + 0x1000, cap=8, out=C):
        return lib.gsort_dispatch_rows(x, dtype, tokens, width, stride, pos, k, rows, cap, out, None)

    assert dispatch(cap=0) == OK
    for bad in (dict(dtype=5), dict(tokens=-1), dict(width=0), dict(stride=7), dict(k=0), dict(cap=-1), dict(x=None), dict(pos=None),
                dict(rows=None), dict(out=None), dict(out=A + 16)):
        assert dispatch(**bad) == EINVAL, bad
    assert dispatch(tokens=1 << 29, k=4) == ETOOBIG and dispatch(cap=1 << 30) == ETOOBIG and dispatch(width=1 << 30, stride=1 << 30) == ETOOBIG
    assert dispatch(x=A + 2) == EALIGN and dispatch(out=C + 1) == EALIGN and dispatch(pos=B + 2) == EALIGN

    def combine(y=A, cap=8, width=8, stride=8, w=B, pos=B + 0x1000, tokens=4, k=2, out=C):
        return lib.gsort_combine_rows(y, 1, cap, width, stride, w, pos, tokens, k, out, None)

    assert combine(tokens=0) == OK
    for bad in (dict(y=None), dict(pos=None), dict(out=None), dict(out=A), dict(out=B), dict(stride=4), dict(k=0)):
        assert combine(**bad) == EINVAL, bad
    assert combine(w=B + 2) == EALIGN

    def back(d=A, y=A + 0x1000, w=B, pos=B + 0x1000, rows=B + 0x2000, dy=C, dw=D, tokens=4, cap=8):
        return lib.gsort_combine_rows_backward(d, 2, tokens, 8, 8, y, cap, 8, w, pos, 2, rows, dy, dw, None)

    assert back(tokens=0, cap=0) == OK
    for bad in (dict(d=None), dict(y=None), dict(w=None), dict(pos=None), dict(rows=None), dict(dy=None), dict(dw=None),
                dict(dy=A), dict(dw=B), dict(dw=C + 16)):
        assert back(**bad) == EINVAL, bad
    assert back(dw=D + 2) == EALIGN


def test_logprobs_argument_errors(lib):
    def call(x=A, dtype=0, rows=4, vocab=16, stride=16, t=B, tb=8, top=0, lp=C, h=C + 0x100, st=C + 0x200, tv=None, ti=None):
        return lib.gsort_token_logprobs(x, dtype, rows, vocab, stride, t, tb, top, lp, h, st, tv, ti, None)

    assert call(rows=0) == OK
    for bad in (dict(dtype=7), dict(rows=-1), dict(vocab=0, stride=0), dict(stride=15), dict(tb=2), dict(top=-1), dict(t=None), dict(lp=None),
                dict(x=None), dict(st=None), dict(top=3), dict(top=3, tv=D), dict(lp=A), dict(h=C), dict(top=3, tv=D, ti=D + 4)):
        assert call(**bad) == EINVAL, bad
    assert call(top=33, tv=D, ti=D + 0x1000) == ETOOBIG and call(rows=(1 << 28) + 1) == ETOOBIG and call(vocab=1 << 30, stride=1 << 30) == ETOOBIG
    for bad in (dict(x=A + 1), dict(t=B + 4), dict(lp=C + 2), dict(st=C + 0x204), dict(top=3, tv=D + 1, ti=D + 0x1000)):
        assert call(**bad) == EALIGN, bad

    def back(dl=A, dh=A + 0x100, x=B, stride=16, t=A + 0x200, h=A + 0x300, st=A + 0x400, out=C, gstride=16, rows=4):
        return lib.gsort_token_logprobs_backward(dl, dh, x, 1, rows, 16, stride, t, 8, h, st, out, gstride, None)

    assert back(rows=0) == OK
    for bad in (dict(t=None), dict(x=None), dict(h=None), dict(st=None), dict(out=None), dict(out=B + 4), dict(out=B, gstride=17),
                dict(out=A), dict(gstride=15)):
        assert back(**bad) == EINVAL, bad
    assert back(out=C + 1) == EALIGN and back(st=A + 0x404) == EALIGN


def test_torch_wrappers_refuse_before_the_device():
    """Wrong types, shapes and devices are found without a GPU."""
    import torch

    import bitonic_networks_gb300 as gs
    x, e = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    g = gs.ExpertGroups(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), e)
    r = gs.TokenLogprobs(torch.zeros(4), torch.zeros(4), None, None, torch.zeros(4, 2))
    for call in (lambda: gs.route_experts(x, 2), lambda: gs.route_experts_backward(torch.zeros(4, 2), x, e),
                 lambda: gs.group_by_expert(e, 8), lambda: gs.dispatch_rows(x, g), lambda: gs.combine_rows(torch.zeros(8, 8), g),
                 lambda: gs.token_logprobs(x), lambda: gs.token_logprobs_backward(None, None, x, None, r)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: gs.route_experts(x.double(), 2), lambda: gs.route_experts([[1.0]], 2), lambda: gs.group_by_expert(e, "8"),
                 lambda: gs.token_logprobs(x.int())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        gs.group_by_expert(e, 2 ** 40)
