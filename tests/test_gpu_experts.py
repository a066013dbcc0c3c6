"""Grouping by expert and the row moves on the GPU: integers bit for bit, sums
against 64-bit forms.  Tolerances, fixed beforehand: a combined row adds k
products in 32 bits (k * 2^-24 of their absolute sum); a weight's gradient adds
at most width / 128 products per thread and 7 levels of a tree; each stored
value is rounded once to its type."""
import numpy as np
import pytest
import torch

import bitonic_networks_gb300 as gs
from bitonic_networks_gb300 import _lib
from model_ref import DTYPES, TINY, UNIT, group_ref, strided

pytestmark = pytest.mark.gpu


def chosen(tokens, k, experts, seed, drop=0.0, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(tokens, experts, generator=g) + skew * torch.rand(experts, generator=g)
    e = torch.argsort(x, 1, descending=True)[:, :k].to(torch.int32)
    if drop:
        e[torch.rand(tokens, k, generator=g) < drop] = -1
    return e.cuda()


def check_group(e, experts, align):
    g = gs.group_by_expert(e, experts, align=align)
    assert g.rows.numel() == gs.group_capacity(e.numel(), experts, align)
    for got, want in zip(g, group_ref(e, experts, align, g.rows.numel())):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), want)
    return g


@pytest.mark.parametrize("pairs", [1, 2, 31, 32, 33, 127, 128, 129, 4095, 4096, 4097, 8192, 50_001, 148 * 4096,
                                   148 * 4096 + 1, 1_300_003])
@pytest.mark.parametrize("experts,align", [(1, 1), (2, 128), (60, 1), (256, 16), (1000, 7), (1024, 1)])
def test_group(pairs, experts, align):
    g = torch.Generator().manual_seed(pairs + experts)
    e = torch.randint(0, experts, (pairs, 1), generator=g, dtype=torch.int32)
    e = torch.where(torch.rand(pairs, 1, generator=g) < 0.3, e // 7, e)     # some experts are busier
    check_group(e.cuda(), experts, align)


def test_group_drops_what_is_no_expert():
    for tokens in (1, 700, 30_000):
        e = chosen(tokens, 4, 64, tokens, drop=0.4)
        e[0] = torch.tensor([64, -2 ** 31, 2 ** 31 - 1, 63], dtype=torch.int32)
        check_group(e, 64, 16)
    check_group(torch.full((999, 3), -1, dtype=torch.int32).cuda(), 8, 4)
    check_group(torch.full((20_000, 1), 5, dtype=torch.int32).cuda(), 8, 128)     # one expert takes all


def test_group_of_nothing():
    g = gs.group_by_expert(torch.empty(0, 8, dtype=torch.int32).cuda(), 16, align=128)
    assert g.rows.numel() == 0 and (g.offsets == 0).all() and (g.counts == 0).all() and g.positions.shape == (0, 8)
    x = torch.empty(0, 32).cuda()
    assert gs.dispatch_rows(x, g).shape == (0, 32)
    assert gs.combine_rows(torch.empty(0, 32).cuda(), g).shape == (0, 32)
    d_y, d_w = gs.combine_rows_backward(x, torch.empty(0, 32).cuda(), g, torch.empty(0, 8).cuda())
    assert d_y.shape == (0, 32) and d_w.shape == (0, 8)


def test_group_workspace_may_hold_anything():
    e = chosen(20_000, 4, 100, 1)
    ws = torch.full((gs.group_workspace_bytes(80_000, 100),), 0xAB, dtype=torch.uint8, device="cuda")
    a, b = gs.group_by_expert(e, 100, workspace=ws), gs.group_by_expert(e, 100)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(gs.GsortError):
        gs.group_by_expert(e, 100, workspace=ws[:256])


def rows64(t):
    return t.double().cpu().numpy()


def check_rows(x, y, d_out, groups, w, k):
    """Every move against 64 bits."""
    dtype, width = x.dtype, x.shape[1]
    rows, pos = groups.rows.cpu().numpy(), groups.positions.cpu().numpy()
    held = rows >= 0
    got = gs.dispatch_rows(x, groups)
    want = np.zeros(got.shape)
    want[held] = rows64(x)[rows[held] // k]
    assert np.array_equal(rows64(got), want)

    y64, d64, w64 = rows64(y), rows64(d_out), rows64(w)
    there = pos >= 0
    safe = np.maximum(pos, 0)
    for weights, ww in ((w, w64), (None, np.ones_like(w64))):
        got = gs.combine_rows(y, groups, weights)
        parts = np.where(there[:, :, None], ww[:, :, None] * y64[safe], 0.0) if len(y64) else np.zeros((len(pos), k, width))
        want, size = parts.sum(1), np.abs(parts).sum(1)
        assert (np.abs(rows64(got) - want) <= (k + 1) * 2.0 ** -24 * size + UNIT[dtype] * np.abs(want) + TINY[dtype]).all()

    d_y, d_w = gs.combine_rows_backward(d_out, y, groups, w)
    want = np.zeros(d_y.shape)
    want[held] = w64.reshape(-1)[rows[held], None] * d64[rows[held] // k]
    # the product is rounded to 32 bits and then to the type
    assert (np.abs(rows64(d_y) - want) <= (UNIT[dtype] + 2.0 ** -23) * np.abs(want) + TINY[dtype]).all()
    parts = np.where(there[:, :, None], y64[safe] * d64[:, None, :], 0.0)
    assert (np.abs(rows64(d_w) - parts.sum(2)) <= (width / 128 + 16) * 2.0 ** -24 * np.abs(parts).sum(2) + 1e-37).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [1, 2, 3, 4, 8, 12, 100, 129, 1001, 2048])
def test_rows(dtype, width):
    for tokens, k, experts, align, drop in ((1, 1, 4, 1, 0.0), (3, 8, 16, 16, 0.0), (130, 5, 12, 8, 0.3), (37, 32, 40, 1, 0.0)):
        e = chosen(tokens, k, experts, width, drop)
        groups = gs.group_by_expert(e, experts, align=align)
        g = torch.Generator().manual_seed(width)
        x, d = (torch.randn(tokens, width, generator=g).to(dtype).cuda() for _ in range(2))
        y = torch.randn(groups.rows.numel(), width, generator=g).to(dtype).cuda()
        check_rows(x, y, d, groups, torch.randn(tokens, k, generator=g).cuda(), k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [5, 33, 136, 515, 1001])
def test_rows_of_many_pairs(dtype, width):
    """Enough pairs that each has a warp or less; more tokens than a CTA holds."""
    e = chosen(1700, 3, 7, width, 0.1)
    groups = gs.group_by_expert(e, 7, align=32)
    g = torch.Generator().manual_seed(width)
    x, d = (torch.randn(1700, width, generator=g).to(dtype).cuda() for _ in range(2))
    y = torch.randn(groups.rows.numel(), width, generator=g).to(dtype).cuda()
    check_rows(x, y, d, groups, torch.randn(1700, 3, generator=g).cuda(), 3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,off", [(1, 0), (0, 1), (8, 0), (4, 4), (2, 2)])
def test_strided_and_unaligned_rows(dtype, pad, off):
    e = chosen(50, 4, 10, 2, 0.2)
    groups = gs.group_by_expert(e, 10, align=4)
    g = torch.Generator().manual_seed(3)
    x, d = (torch.randn(50, 136, generator=g).to(dtype).cuda() for _ in range(2))
    y = torch.randn(groups.rows.numel(), 136, generator=g).to(dtype).cuda()
    w = torch.randn(50, 4, generator=g).cuda()
    check_rows(strided(x, pad, off), strided(y, pad, off), strided(d, pad, off), groups, w, 4)
    check_rows(strided(x, pad, off), y, d, groups, w, 4)


def test_masked_tokens_keep_their_contents_out():
    """NaN and infinities in rows that no pair holds, and in dropped tokens, reach nothing."""
    e = chosen(40, 4, 8, 5)
    e[7] = -1
    groups = gs.group_by_expert(e, 8, align=16)
    g = torch.Generator().manual_seed(3)
    y = torch.randn(groups.rows.numel(), 64, generator=g).cuda()
    y[groups.rows < 0] = float("nan")
    x = torch.randn(40, 64, generator=g).cuda()
    x[7] = float("inf")
    w = torch.rand(40, 4, generator=g).cuda()
    w[7] = float("nan")
    out = gs.combine_rows(y, groups, w)
    assert torch.isfinite(out).all() and (out[7] == 0).all()
    assert torch.isfinite(gs.dispatch_rows(x, groups)).all()
    d_y, d_w = gs.combine_rows_backward(x, y, groups, w)
    assert torch.isfinite(d_y).all() and (d_w[7] == 0).all() and torch.isfinite(d_w).all()


def test_a_layout_without_tokens_is_zero():
    """Rows of the layout that nothing was sent to, from no token at all."""
    empty = gs.ExpertGroups(torch.zeros(5, dtype=torch.int32).cuda(), torch.zeros(4, dtype=torch.int32).cuda(),
                            torch.full((70,), -1, dtype=torch.int32).cuda(), torch.empty(0, 2, dtype=torch.int32).cuda())
    for width in (8, 33):
        assert (gs.dispatch_rows(torch.empty(0, width).cuda(), empty) == 0).all()
        d_y, d_w = gs.combine_rows_backward(torch.empty(0, width).cuda(), torch.ones(70, width).cuda(), empty, torch.empty(0, 2).cuda())
        assert (d_y == 0).all() and d_w.shape == (0, 2)
        assert gs.combine_rows(torch.ones(70, width).cuda(), empty).shape == (0, width)


def test_all_pairs_dropped():
    e = torch.full((9, 3), -1, dtype=torch.int32).cuda()
    groups = gs.group_by_expert(e, 4, align=4)
    for width in (8, 33):
        x, y = torch.ones(9, width).cuda(), torch.ones(groups.rows.numel(), width).cuda()
        assert (gs.dispatch_rows(x, groups) == 0).all() and (gs.combine_rows(y, groups) == 0).all()
        d_y, d_w = gs.combine_rows_backward(x, y, groups, torch.ones(9, 3).cuda())
        assert (d_y == 0).all() and (d_w == 0).all()


def test_positions_outside_the_layout_take_no_part():
    e = chosen(16, 2, 4, 6)
    g = gs.group_by_expert(e, 4)
    positions = g.positions.clone()
    positions[3, 0], positions[4, 1] = 32, 2 ** 31 - 1
    bad = g._replace(positions=positions)
    y = torch.ones(32, 8).cuda()
    assert gs.combine_rows(y, bad)[3:5].tolist() == [[1.0] * 8] * 2
    assert gs.dispatch_rows(torch.ones(16, 8).cuda(), bad).shape == (32, 8)


def test_offsets_beyond_32_bits():
    """A layout of more than 2^32 bytes and 2^31 elements."""
    tokens, k, width = 5000, 8, 65536
    e = chosen(tokens, k, 16, 7)
    groups = gs.group_by_expert(e, 16)
    x = torch.randn(tokens, 1, device="cuda").expand(tokens, width).to(torch.bfloat16).contiguous()
    out = gs.dispatch_rows(x, groups)
    assert out.numel() > 2 ** 31
    pair = groups.rows.long()
    assert torch.equal(out[:, -1], x[pair // k, -1]) and torch.equal(out[:, 0], x[pair // k, 0])
    back = gs.combine_rows(out, groups, torch.full((tokens, k), 0.125, device="cuda"))
    assert torch.equal(back, x)                # eight equal rows, an eighth each: exact
    d_y, d_w = gs.combine_rows_backward(x, out, groups, torch.ones(tokens, k, device="cuda"))
    assert torch.equal(d_y[:, -1], out[:, -1])
    want = x[:, :1].double() ** 2 * width
    assert torch.allclose(d_w.double(), want.expand(-1, k), rtol=1e-4)


def test_gradients_against_differences():
    """<d_out, combine(y, w)> and <d_rows, dispatch(x)> are bilinear: exact differences."""
    e = chosen(21, 3, 9, 8, 0.2)
    groups = gs.group_by_expert(e, 9, align=2)
    g = torch.Generator().manual_seed(1)
    n = groups.rows.numel()
    y, dy = torch.randn(n, 40, generator=g).cuda(), torch.randn(n, 40, generator=g).cuda()
    w, dw = torch.randn(21, 3, generator=g).cuda(), torch.randn(21, 3, generator=g).cuda()
    d = torch.randn(21, 40, generator=g).cuda()

    def loss(yy, ww):
        return float((gs.combine_rows(yy, groups, ww).double() * d.double()).sum())

    d_y, d_w = gs.combine_rows_backward(d, y, groups, w)
    by_y, by_w = float((d_y.double() * dy.double()).sum()), float((d_w.double() * dw.double()).sum())
    # about 2500 products of size 1, each off by a few 2^-24
    assert abs(loss(y + dy, w) - loss(y - dy, w) - 2 * by_y) < 2e-3
    assert abs(loss(y, w + dw) - loss(y, w - dw) - 2 * by_w) < 2e-3
    x = torch.randn(21, 40, generator=g).cuda()
    through = float((gs.dispatch_rows(x, groups).double() * dy.double()).sum())
    assert abs(through - float((gs.combine_rows(dy, groups).double() * x.double()).sum())) < 1e-3


def test_refusals():
    e = chosen(8, 2, 4, 1)
    groups = gs.group_by_expert(e, 4)
    x, y, w = torch.zeros(8, 16).cuda(), torch.zeros(16, 16).cuda(), torch.zeros(8, 2).cuda()
    for bad in (lambda: gs.group_by_expert(e.long(), 4), lambda: gs.dispatch_rows(x.double(), groups),
                lambda: gs.combine_rows(y, groups, w.half()), lambda: gs.combine_rows_backward(x, y.half(), groups, w)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: gs.group_by_expert(e.cpu(), 4), lambda: gs.group_by_expert(e.view(-1), 4),
                lambda: gs.dispatch_rows(x[:7], groups), lambda: gs.combine_rows(y[:15], groups),
                lambda: gs.combine_rows(y, groups, w.view(2, 8)), lambda: gs.dispatch_rows(x.t(), groups),
                lambda: gs.combine_rows_backward(x[:, :8], y, groups, w), lambda: gs.dispatch_rows(x.cpu(), groups)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        gs.group_by_expert(e, 2 ** 32 + 4)
    for experts, align in ((0, 1), (1025, 1), (4, 0), (-1, 1), (1024, 2 ** 31 - 1)):
        with pytest.raises(gs.GsortError):
            gs.group_by_expert(e, experts, align=align)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [1, 33, 136, 1001])
def test_rows_of_dropped_positions_are_zero(dtype, width):
    """A pair whose position was taken away (or moved outside the layout) holds no
    row: its row of the layout is written as zeros, not left as it was."""
    lib, code = _lib.load(), DTYPES.index(dtype)
    tokens, k, experts = 300, 3, 8
    groups = gs.group_by_expert(chosen(tokens, k, experts, width), experts, align=16)
    positions = groups.positions.clone()
    gone = torch.rand(tokens, k, generator=torch.Generator().manual_seed(5)).cuda() < 0.3
    rows = positions[gone].long()
    positions[gone] = -1
    positions[0, 0] = groups.rows.numel()
    rows = torch.cat([rows, groups.positions[0, :1].long()])
    capacity = groups.rows.numel()
    g = torch.Generator().manual_seed(3)
    x, y = torch.randn(tokens, width, generator=g).to(dtype).cuda(), torch.randn(capacity, width, generator=g).to(dtype).cuda()
    w = torch.randn(tokens, k, generator=g).cuda()
    whole = gs.dispatch_rows(x, groups)
    d_whole, _ = gs.combine_rows_backward(x, y, groups, w)
    whole[rows], d_whole[rows] = 0.0, 0.0
    stream = torch.cuda.current_stream().cuda_stream
    out, d_y, d_w = torch.full_like(y, 7.0), torch.full_like(y, 7.0), torch.full_like(w, 7.0)
    assert lib.gsort_dispatch_rows(x.data_ptr(), code, tokens, width, width, positions.data_ptr(), k, groups.rows.data_ptr(), capacity,
                                   out.data_ptr(), stream) == 0
    assert lib.gsort_combine_rows_backward(x.data_ptr(), code, tokens, width, width, y.data_ptr(), capacity, width, w.data_ptr(),
                                           positions.data_ptr(), k, groups.rows.data_ptr(), d_y.data_ptr(), d_w.data_ptr(), stream) == 0
    assert torch.equal(out, whole) and torch.equal(d_y, d_whole)
    assert (d_w[gone] == 0).all() and d_w[0, 0] == 0
