"""gradient_norm and clip_gradients against 64-bit sums: many tensors of odd sizes and
mixed types, numbers whose squares leave the 32-bit range, in place, refusals."""
import math
import threading

import pytest
import torch

import bitonic_networks_gb300 as gs
from model_ref import DTYPES, TINY, UNIT
from vocab_ref import U32, f32

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# a thread sums at most 128 squares in 8 chains of 16, then the 8: 24 roundings of
# numbers of one sign, half of that under the root; the rest is 64-bit, and the norm rounds once
NORM = 14 * U32


def norm64(tensors):
    return math.sqrt(float(torch.stack([(t.double() ** 2).sum() for t in tensors]).sum()))


def make(sizes, dtypes=None, seed=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dtype = (dtypes or DTYPES)[i % len(dtypes or DTYPES)]
        buffer = torch.randn(n + off, generator=g, device="cuda").to(dtype)
        out.append(buffer[off:] if off else buffer)
    return out


def check_clip(tensors, max_norm, scale=1.0, out=None):
    before = [t.clone() for t in tensors]
    norm = abs(f32(scale)) * norm64(tensors)
    r = gs.clip_gradients(tensors, max_norm, scale=scale, out=out)
    assert abs(float(r.norm) - norm) <= NORM * norm and r.norm.dtype == torch.float32 and r.norm.dim() == 0
    by = f32(scale) * min(1.0, f32(max_norm) / norm if norm > 0 else 1.0)
    assert len(r.gradients) == len(tensors)
    for x, y in zip(before, r.gradients):
        assert y.dtype == x.dtype and y.shape == x.shape and y.stride() == x.stride()
    for dtype in {x.dtype for x in before}:
        want, got = (torch.cat([t.flatten() for t in ts if t.dtype == dtype]).double() for ts in (before, r.gradients))
        want = want * by
        # the norm's error, the factor's and the product's roundings, and the type's
        assert bool(((got - want).abs() <= want.abs() * (NORM + 3 * U32 + UNIT[dtype]) + TINY[dtype]).all())
    if out is None:
        assert all(torch.equal(x, y) for x, y in zip(before, tensors))
    else:
        assert all(x is y for x, y in zip(out, r.gradients))
    return r


SIZES = {"one": [1], "empty among them": [0, 5, 0], "few": [7, 4096, 33, 100001, 2], "vectors": [8, 16, 4, 64], "33": [1000 + i for i in range(33)],
         "1000": [13 * i % 400 for i in range(1000)], "1001": [37] * 1001, "2500": [1 + 7 * i % 90 for i in range(2500)], "large": [3_000_001, 20_000_003]}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("off", [0, 1, 3])
def test_norm_and_clipping(name, off):
    for dtypes in (None, *([d] for d in DTYPES if len(SIZES[name]) < 50)):
        tensors = make(SIZES[name], dtypes, off=off)
        norm = norm64(tensors)
        got = gs.gradient_norm(tensors)
        assert got.dtype == torch.float32 and got.dim() == 0 and abs(float(got) - norm) <= NORM * norm
        assert torch.equal(got, gs.gradient_norm(tuple(tensors)))          # the same order of sums
        for max_norm, scale in ((0.25 * norm, 1.0), (2.0 * norm, 1.0), (0.5 * norm, -0.75), (INF, 0.3)):
            check_clip(tensors, max_norm, scale)
        check_clip(tensors, 0.3 * norm, out=make(SIZES[name], dtypes, seed=1, off=off))
        check_clip(tensors, 0.3 * norm, out=make(SIZES[name], dtypes, seed=1, off=2 - off % 2))     # lying differently
        mine = [t.clone() for t in tensors]
        versions = [t._version for t in mine]
        check_clip(mine, 0.3 * norm, out=mine)
        assert all(t._version > v for t, v in zip(mine, versions))


def test_what_is_not_clipped_stays_bit_for_bit():
    tensors = make([1000, 77], [torch.float32, torch.bfloat16])
    tensors[0][3] = -0.0
    tensors[1][5] = 1e-40
    norm = norm64(tensors)
    mine = [t.clone() for t in tensors]
    for out in (mine, [torch.full_like(t, 9.0) for t in tensors]):
        r = gs.clip_gradients(mine, 1.5 * norm, out=out)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r.gradients, tensors))


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-40, 1e-45])
def test_squares_beyond_32_bits(value):
    t = torch.full((70001,), value, device="cuda")
    v = float(t[0])
    want = v * math.sqrt(70001)
    got = float(gs.gradient_norm([t]))
    assert got == INF if want > 3.4e38 else abs(got - want) <= NORM * want + 1e-45
    # the large ones beside the small ones, and clipping to 1
    both = [t, torch.full((5000,), 1e-20, device="cuda"), torch.zeros(100, device="cuda")]
    norm = norm64(both)
    r = gs.clip_gradients(both, norm / 4 if norm < 1e38 else 1e37)
    by = 0.25 if norm < 1e38 else f32(1e37) / norm
    # the factor 0.25 of an f32 norm / 4: rounded by the caller
    assert torch.allclose(r.gradients[0].double(), t.double() * by, rtol=4e-6, atol=1e-45)
    assert bool((r.gradients[2] == 0).all())


def test_bf16_beyond_32_bits():
    t = torch.full((5000,), 1e30, dtype=torch.bfloat16, device="cuda")
    want = float(t[0]) * math.sqrt(5000)
    assert abs(float(gs.gradient_norm([t])) - want) <= NORM * want
    t = torch.full((5000,), 2.0 ** -24, dtype=torch.float16, device="cuda")
    assert abs(float(gs.gradient_norm([t])) - 2.0 ** -24 * math.sqrt(5000)) <= NORM * 2.0 ** -17


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinities(dtype):
    x, y = torch.ones(3000, dtype=dtype, device="cuda"), torch.ones(50, device="cuda")
    x[1234] = NAN
    r = gs.clip_gradients([x, y], 1.0)
    assert math.isnan(float(r.norm)) and all(bool(t.isnan().all()) for t in r.gradients) and math.isnan(float(gs.gradient_norm([y, x])))
    x[1234] = -INF
    r = gs.clip_gradients([x, y], 1.0)
    assert float(r.norm) == INF and bool((r.gradients[1] == 0).all()) and bool(r.gradients[0][1234].isnan()) and int((r.gradients[0] != 0).sum()) == 1
    r = gs.clip_gradients([x, y], INF, scale=0.5)
    assert float(r.norm) == INF and bool((r.gradients[1] == 0.5).all()) and bool(r.gradients[0][1234].isneginf())


def test_zeros_and_a_limit_of_zero():
    x = torch.zeros(5000, device="cuda")
    r = gs.clip_gradients([x], 0.0)
    assert float(r.norm) == 0.0 and bool((r.gradients[0] == 0).all())
    r = gs.clip_gradients([x + 2.0], 0.0)
    assert bool((r.gradients[0] == 0).all()) and float(r.norm) > 0
    empty = [torch.zeros(0, device="cuda")]
    assert float(gs.gradient_norm(empty)) == 0.0 and float(gs.clip_gradients(empty, 1.0).norm) == 0.0


def test_dense_tensors_in_any_order_of_strides():
    x = torch.randn(40, 50, 6, device="cuda")
    for t in (x.t() if x.dim() == 2 else x.permute(2, 0, 1), x.transpose(0, 1), torch.randn(30, 7, device="cuda").t(),
              torch.randn(2, 5, 4, 3, device="cuda").to(memory_format=torch.channels_last)):
        check_clip([t, x], 1.0)
        check_clip([t, x], 1.0, out=[torch.empty_like(t), torch.empty_like(x)])


def test_any_sequence_of_tensors():
    x, y = torch.randn(100, device="cuda"), torch.randn(40, device="cuda")
    want = gs.clip_gradients([x, y], 1.0)
    for make_list in (tuple, iter, lambda ts: (t for t in ts)):
        got = gs.clip_gradients(make_list([x, y]), 1.0, out=make_list([torch.empty_like(x), torch.empty_like(y)]))
        assert isinstance(got.gradients, list) and torch.equal(got.norm, want.norm) and all(torch.equal(a, b) for a, b in zip(got.gradients, want.gradients))
    with torch.inference_mode():
        z = x.clone()
        assert gs.clip_gradients([z], 1.0, out=[z]).gradients[0] is z


def test_lists_that_another_thread_changes():
    kept = [torch.randn(64, device="cuda") for _ in range(200)]
    want = gs.clip_gradients(kept, 1.0)
    gradients, out, stop = list(kept), [torch.empty_like(t) for t in kept], threading.Event()
    whole_out = list(out)

    def change():
        while not stop.is_set():
            for items, whole in ((gradients, kept), (out, whole_out)):
                items.clear()
                items.extend(whole)

    thread = threading.Thread(target=change)
    thread.start()
    try:
        for k in range(300):
            try:
                got = gs.clip_gradients(gradients, 1.0, out=out if k % 2 else None)
            except ValueError:          # the call came upon an empty list
                continue
            assert len(got.gradients) == 200 and torch.equal(got.norm, want.norm) and torch.equal(got.gradients[-1], want.gradients[-1])
    finally:
        stop.set()
        thread.join()


def test_the_same_tensor_twice():
    x = torch.randn(1000, device="cuda")
    assert abs(float(gs.gradient_norm([x, x])) - math.sqrt(2) * norm64([x])) <= NORM * 2 * norm64([x])
    check_clip([x, x], 1.0)                                     # outputs of their own
    with pytest.raises(gs.GsortError):
        gs.clip_gradients([x, x], 1.0, out=[x, x])
    with pytest.raises(gs.GsortError):
        gs.clip_gradients([x, x.clone()], 1.0, out=[x, x])


def test_more_elements_than_32_bits():
    t = torch.zeros((1 << 32) + 100, dtype=torch.bfloat16, device="cuda")
    t[-1], t[0], t[1 << 31] = 4.0, 2.0, 4.0
    assert float(gs.gradient_norm([t])) == 6.0
    gs.clip_gradients([t], 3.0, out=[t])
    assert t[[-1, 0, 1 << 31]].tolist() == [2.0, 1.0, 2.0] and float(gs.gradient_norm([t])) == 3.0


def test_refusals():
    x, y = torch.randn(100, device="cuda"), torch.randn(40, device="cuda")
    for call in (lambda: gs.gradient_norm(x.double()), lambda: gs.gradient_norm([x, None]), lambda: gs.gradient_norm([x.int()]), lambda: gs.gradient_norm(3),
                 lambda: gs.clip_gradients([x], None), lambda: gs.clip_gradients([x], 1.0, out=3), lambda: gs.clip_gradients([x], 1.0, out=[None])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: gs.gradient_norm([]), lambda: gs.clip_gradients([], 1.0), lambda: gs.gradient_norm([x, y.cpu()]), lambda: gs.gradient_norm([x[::2]]),
                 lambda: gs.gradient_norm([x.expand(3, 100)]), lambda: gs.gradient_norm([x.to_sparse()]), lambda: gs.clip_gradients([x], 1.0, out=[]), lambda: gs.clip_gradients([x], 1.0, out=[y]),
                 lambda: gs.clip_gradients([x], 1.0, out=[x.half()]), lambda: gs.clip_gradients([x.view(10, 10)], 1.0, out=[torch.empty(10, 10, device="cuda").t()])):
        with pytest.raises(ValueError):
            call()
    buffer = torch.randn(300, device="cuda")
    for call in (lambda: gs.clip_gradients([x], -1.0), lambda: gs.clip_gradients([x], NAN), lambda: gs.clip_gradients([x], 1.0, scale=INF),
                 lambda: gs.clip_gradients([buffer[:100]], 1.0, out=[buffer[50:150]]), lambda: gs.clip_gradients([x, x.clone()], 1.0, out=[buffer[:100], buffer[60:160]]),
                 lambda: gs.clip_gradients([buffer[:100], buffer[100:200]], 1.0, out=[buffer[100:200], buffer[:100]])):
        with pytest.raises(gs.GsortError):
            call()
    z = torch.randn(5, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        gs.gradient_norm([z])
    with pytest.raises(RuntimeError, match="no gradient"):
        gs.clip_gradients([z], 1.0)
    with torch.no_grad():
        gs.clip_gradients([z], 1.0, out=[z])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 1e-5])
@pytest.mark.parametrize("n", [70001, 3])
def test_norms_far_beyond_the_limit(dtype, max_norm, n):
    """The factor is below the smallest normal 32-bit number: it must not lose bits, or become 0."""
    g = torch.Generator(device="cuda").manual_seed(n)
    sign = torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)
    t = ((torch.rand(n, generator=g, device="cuda") * 0.25 + 0.75) * 3.3e38 * sign).to(dtype)
    by = f32(max_norm) / norm64([t])
    assert by < 2.0 ** -126
    # squares beyond the 32-bit range are summed in 64 bits, so the factor is; the product rounds to 32 bits, then to the type
    want = t.double() * by
    error = want.abs() * (UNIT[dtype] + 2 * U32)
    for out in (None, [torch.empty_like(t)], [torch.empty(n + 1, dtype=dtype, device="cuda")[1:]], [t]):
        r = gs.clip_gradients([t], max_norm, out=out)
        assert float(r.norm) == INF         # beyond 32 bits
        assert bool(((r.gradients[0].double() - want).abs() <= error).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("value", [None, 1.1, 0.7, 1 / 3, 0.013])
@pytest.mark.parametrize("n", [3, 4096, 16384, 1_000_003, 30_000_000])
def test_the_norm_is_as_near_as_a_steps_sums_allow(dtype, value, n):
    """Of a step a thread has 4 vectors: 4 chains of 4 products (f32) or 8 (16 bits), joined by 2 additions: 6 or 10 roundings
    of numbers of one sign, half of that under the root.  All else is 64-bit, and the norm rounds once.  Equal numbers
    round alike in every chain, so that errors do not cancel."""
    if value is None:
        t = torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").add_(0.5).to(dtype)
    else:
        t = torch.full((n,), value, device="cuda").to(dtype)
    want = norm64([t])
    near = ((3 if dtype == torch.float32 else 5) + 1) * U32 * 1.0001         # the rest is of second order
    assert abs(float(gs.gradient_norm([t])) - want) <= near * want
    assert abs(float(gs.clip_gradients([t], 1.0).norm) - want) <= near * want


@pytest.mark.parametrize("count", [3, 1200])
def test_replays_on_smaller_gradients(count):
    """Each replay gives the norm of what is there then, not of what was there before."""
    tensors = [torch.randn(5000, device="cuda") for _ in range(count)]
    out = [torch.empty_like(t) for t in tensors]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gs.clip_gradients(tensors, 1.0, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = gs.clip_gradients(tensors, 1.0, out=out)
    for by in (1.0, 1e-3, 0.0, float("nan"), 1.0):
        for t in tensors:
            t.normal_().mul_(by)
        graph.replay()
        want = gs.clip_gradients(tensors, 1.0)
        assert torch.equal(held.norm.view(torch.int32), want.norm.view(torch.int32))
        assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(out, want.gradients))
