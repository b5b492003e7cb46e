"""The global gradient norm and clipping (GPU) against float64 evaluations.

A thread adds up to 16 squares a chain in fp32 and joins four or eight chains: its sum is off by 2^-19 of itself, a sum of
squares, so the norm by 2^-20, and by 2^-24 from its rounding.  A scaled value is off by the factor's error
and two roundings more (2^-23), and half a step of its type (bf16 2^-8, f16 2^-11, subnormal steps besides)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
NORM = 2.0 ** -19
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def _check(wb, grads, max_norm, f32_out=False):
    want = _norm(grads)
    k = max_norm / want if want > max_norm else 1.0
    before = [g.clone() for g in grads]
    got = wb.grad_norm(grads)
    assert abs(float(got) - want) <= NORM * want
    outs = [torch.full_like(g, math.nan, dtype=torch.float32 if f32_out else g.dtype) for g in grads]
    again = wb.clip_grad_norm(grads, max_norm, out=outs)
    assert torch.equal(got, again) and got.shape == ()
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    norm = wb.clip_grad_norm(grads, max_norm)
    assert torch.equal(got, norm) and wb.check_device_error() == 0
    for g, b, o in zip(grads, before, outs):
        exact = b.double() * k
        for t in (g, o):
            off = (NORM + 2.0 ** -22 + HALF[t.dtype]) * exact.abs() + TINY[t.dtype] if k < 1 else torch.zeros_like(exact)
            assert bool(((t.double() - exact).abs() <= off).all())
        if not f32_out:
            assert torch.equal(g, o)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shapes", [[(1,)], [(7,)], [(2, 3), (0,), (5,)], [(1283, 387)], [(16384,)], [(16385,), (8191,), (8192,), (8193,)],
                                    [(64,), (1 << 20,), (33,)], [(9, 1001), ()], [(3, 5)] * 97, [(100,)] * 2000])
@pytest.mark.parametrize("max_norm", [0.37, 1e9])
def test_against_float64(wb, kind, shapes, max_norm):
    g = torch.Generator(device=DEV).manual_seed(len(shapes))
    grads = [torch.randn(s, generator=g, device=DEV).to(TYPES[kind]) for s in shapes]
    _check(wb, grads, max_norm, f32_out=len(shapes) % 2 == 1)


def test_mixed_types_orders_and_alignments(wb):
    # views at every element offset of larger buffers, permuted ones, all types in one call; neighbours stay as they are
    g = torch.Generator(device=DEV).manual_seed(1)
    grads, buffers = [], []
    for i, t in enumerate([torch.bfloat16, torch.float16, torch.float32] * 8):
        n = (1, 5, 31, 9000, 40000, 16384 + i)[i % 6]
        buf = torch.randn(n + 16, generator=g, device=DEV).to(t)
        buffers.append((buf, buf.clone(), i % 9, n))
        grads.append(buf[i % 9:i % 9 + n])
    m = torch.randn(40, 30, 20, generator=g, device=DEV)
    grads += [m.permute(2, 0, 1), torch.randn(50, 60, generator=g, device=DEV).half().T]
    _check(wb, grads, 1.25)
    for buf, was, lo, n in buffers:
        assert torch.equal(buf[:lo], was[:lo]) and torch.equal(buf[lo + n:], was[lo + n:])
    # outputs whose 16-byte boundaries lie elsewhere
    src = torch.randn(30001, generator=g, device=DEV).to(torch.bfloat16)
    for shift in range(5):
        dst = torch.zeros(30010, device=DEV)
        wb.clip_grad_norm([src[1:30000]], 1.0, out=[dst[shift:shift + 29999]])
        k = min(1.0, 1.0 / _norm([src[1:30000]]))
        assert bool(((dst[shift:shift + 29999].double() - src[1:30000].double() * k).abs() <= (NORM + 2.0 ** -22) * src[1:30000].double().abs() * k).all())
        assert not dst[:shift].any() and not dst[shift + 29999:].any()


@pytest.mark.parametrize("size", [2.0 ** 126, 2.0 ** 70, 2.0 ** 62, 2.0 ** -62, 2.0 ** -70, 2.0 ** -120, 2.0 ** -133])
@pytest.mark.parametrize("n", [1, 1000, 50000])
def test_the_whole_range_of_the_types(wb, size, n):
    # powers of two, exact: 1 to 50000 of them, beside ordinary and zero values
    for t in (torch.float32, torch.bfloat16):
        big = torch.full((n,), size, device=DEV).to(t)
        want = size * math.sqrt(n)
        got = float(wb.grad_norm([big, torch.zeros(5000, device=DEV)]))
        if want < 3.4e38:
            assert abs(got - want) <= NORM * want + 2.0 ** -149
        else:
            assert got == math.inf
        both = torch.cat([big, torch.ones(3000, device=DEV, dtype=t)])
        want = math.hypot(want, math.sqrt(3000))
        got = float(wb.grad_norm([both]))
        assert (got == math.inf) if want >= 3.4e38 else abs(got - want) <= NORM * want
    assert wb.check_device_error() == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_norm_that_is_not_finite_changes_nothing(wb, bad):
    for t in TYPES.values():
        grads = [torch.randn(20000, device=DEV).to(t), torch.randn(7, device=DEV)]
        grads[0][12345] = bad
        before = [g.clone() for g in grads]
        outs = [torch.zeros_like(g) for g in grads]
        norm = float(wb.clip_grad_norm(grads, 1.0, out=outs))
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
        wb.clip_grad_norm(grads, 1.0)
        for a, b, o in zip(grads, before, outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(o.view(torch.uint8), b.view(torch.uint8))


def test_borders_of_the_factor(wb):
    x = torch.full((4,), 0.5, device=DEV)               # norm 1
    assert float(wb.clip_grad_norm([x], 1.0)) == 1.0 and bool((x == 0.5).all())
    assert float(wb.clip_grad_norm([x], math.inf)) == 1.0 and bool((x == 0.5).all())
    assert float(wb.clip_grad_norm([x], 0.0)) == 1.0 and not x.any()
    assert float(wb.clip_grad_norm([x], 0.0)) == 0.0 and float(wb.grad_norm([torch.zeros(0, device=DEV)])) == 0.0


def test_more_elements_than_32_bits_hold(wb):
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    x[-5:] = 3
    x[0] = 4
    assert abs(float(wb.grad_norm([x])) - math.sqrt(61)) <= NORM * 8
    wb.clip_grad_norm([x], math.sqrt(61) / 2)
    assert bool((x[-5:] == 1.5).all()) and float(x[0]) == 2 and float(x[-6]) == 0


def test_same_bits_side_stream_and_captured(wb):
    g = torch.Generator(device=DEV).manual_seed(2)
    make = lambda: [torch.randn(n, generator=g.manual_seed(5), device=DEV).to(t) for n in (3, 70000, 5001) for t in TYPES.values()]  # noqa: E731
    a, b, c = make(), make(), make()
    n1 = wb.clip_grad_norm(a, 0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n2 = wb.clip_grad_norm(b, 0.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    outs = [torch.empty_like(t) for t in c]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3 = wb.clip_grad_norm(c, 0.5, out=outs)
    for _ in range(2):
        n3.fill_(0)
        graph.replay()
    assert torch.equal(n1, n2) and torch.equal(n1, n3)
    for x, y, z in zip(a, b, outs):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_python_refusals(wb):
    x, y = torch.ones(4, device=DEV), torch.ones(4, device=DEV, dtype=torch.bfloat16)
    for bad in (lambda: wb.grad_norm([x.int()]), lambda: wb.grad_norm([torch.ones(4, 4, device=DEV)[:, :2]]), lambda: wb.grad_norm([None]),
                lambda: wb.grad_norm([x.expand(3, 4)]), lambda: wb.clip_grad_norm([x], 1.0, out=[y]), lambda: wb.clip_grad_norm([x], 1.0, out=[x, x]),
                lambda: wb.clip_grad_norm([y], 1.0, out=[y.half()]), lambda: wb.clip_grad_norm([x], 1.0, out=[x[:2]]),
                lambda: wb.clip_grad_norm([torch.ones(2, 3, device=DEV).T], 1.0, out=[torch.ones(3, 2, device=DEV)])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wb.clip_grad_norm([x, x], 1.0), lambda: wb.clip_grad_norm([x], -1.0), lambda: wb.clip_grad_norm([x], math.nan),
                lambda: wb.clip_grad_norm([x[:3], x[2:]], 1.0), lambda: wb.clip_grad_norm([x[:3]], 1.0, out=[x[1:]])):
        with pytest.raises(wb.WbError):
            bad()
    assert bool((x == 1).all()) and abs(float(wb.grad_norm([x, x])) - math.sqrt(8)) < 1e-5


@pytest.mark.parametrize("max_norm", [2.0 ** -6, 2.0 ** -10, 2.0 ** -20, 2.0 ** -27, 2.0 ** -60, 2.0 ** -100, 2.0 ** -149])
@pytest.mark.parametrize("size", [2.0 ** 119, 2.0 ** 100, 1.7 * 2.0 ** 118])
def test_factors_that_float32_holds_badly_or_not_at_all(wb, size, max_norm):
    # a factor of 2^-114 to 2^-276: exact values are ordinary numbers as long as the gradients are large
    g = torch.Generator(device=DEV).manual_seed(3)
    buf = (size * (1 + torch.rand(20011, generator=g, device=DEV))).to(torch.bfloat16)
    grads = [size * (1 + torch.rand(1000, generator=g, device=DEV)), buf[:3], buf[3:20010], torch.randn(500, generator=g, device=DEV),
             torch.randn(700, generator=g, device=DEV).half(), -size * (1 + torch.rand(9001, generator=g, device=DEV))[1:]]
    _check(wb, grads, max_norm)
    grads = [size * (1 + torch.rand(16400, generator=g, device=DEV)).to(torch.bfloat16), torch.randn(9, generator=g, device=DEV).half(),
             -size * torch.ones(16390, device=DEV)]
    _check(wb, grads, max_norm, f32_out=True)


def test_kernels_counted_of_long_lists(wb):
    # up to 96 tensors a launch of each pass, or 960
    for n, launches in ((1, 2), (96, 2), (97, 2), (960, 2), (961, 4), (2000, 6)):
        grads = [torch.ones(3, device=DEV) for _ in range(n)]
        for clip in (True, False):
            wb.profile_begin()
            try:
                wb.clip_grad_norm(grads, 1.0) if clip else wb.grad_norm(grads)
            finally:
                counts = wb.profile_end()
            assert counts["train.clip"][1] == (launches if clip else launches // 2 + 1), (n, clip)
