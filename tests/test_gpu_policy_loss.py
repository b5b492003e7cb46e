"""The clipped policy loss with its KL term and its gradient (GPU) against float64 evaluations.

A token's ratio e^d is off by 2^-22 (exp) and |d| 2^-24 (the difference's rounding), its product by 2^-24; e^x - 1 by 2^-22 and |x| 2^-24 e^x;
e^x - x - 1 by 2^-20 of itself, and by the rounding of x times its slope.  Sums of n tokens in a sequence are off by (n / 32 + 8) 2^-24
of their terms' magnitude, weights and results by 2^-22."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _data(S, T, seed, per_token=False, empty=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    nll = torch.empty(S, T, device=DEV).exponential_(0.7, generator=g)
    old = nll + 0.3 * torch.randn(S, T, generator=g, device=DEV)
    ref = nll + 0.5 * torch.randn(S, T, generator=g, device=DEV)
    adv = torch.randn(*((S, T) if per_token else (S,)), generator=g, device=DEV)
    labels = torch.randint(0, 50000, (S, T), generator=g, device=DEV)
    labels[torch.rand(S, T, generator=g, device=DEV) < 0.3] = -100
    if empty and S > 2:
        labels[S // 2] = -1
    return nll, old, ref, adv, labels


def _reference(nll, old, ref, adv, labels, lo, hi, beta, per_sequence):
    on = labels >= 0
    n = on.double().sum(1)
    if per_sequence:
        w = torch.where(n > 0, 1 / (n.clamp(min=1) * (n > 0).sum().clamp(min=1)), 0.0)
    else:
        w = (n > 0) / n.sum().clamp(min=1)
    a = (adv if adv.dim() == 2 else adv[:, None].expand_as(nll)).double()
    # what takes no part is out of every expression
    nll, old = torch.where(on, nll, 0).double(), torch.where(on, old, 0).double()
    ref = nll if ref is None else torch.where(on, ref, 0).double()
    a = torch.where(on, a, 0)
    d, x = old - nll, nll - ref
    r = torch.exp(d)
    free = torch.where(a == 0, 0.0, r * a)
    held = torch.where(a == 0, 0.0, r.clamp(1 - lo, 1 + hi) * a)
    clipped = (held < free) & on
    kl = torch.expm1(x) - x
    token = -torch.minimum(free, held) + beta * kl
    grad = torch.where(clipped, 0.0, free) + beta * torch.expm1(x)
    e_r = free.abs() * (2.0 ** -21 + d.abs() * 2.0 ** -23)
    e_em1 = 2.0 ** -22 * torch.expm1(x).abs() + x.abs() * 2.0 ** -23 * torch.exp(x)
    e_kl = 2.0 ** -20 * kl + x.abs() * 2.0 ** -23 * torch.expm1(x).abs() + 2.0 ** -140
    wt = w[:, None] * on
    count = 2.0 ** -24 * (float(n.max()) / 32 + 8) + 2.0 ** -22
    stats = torch.stack([(wt * token).sum(), (wt * kl).sum(), (wt * clipped).sum()])
    e_stats = torch.stack([(wt * (e_r + beta * e_kl)).sum() + count * (wt * (free.abs() + held.abs() + beta * kl)).sum(),
                           (wt * e_kl).sum() + count * (wt * kl).sum(), stats[2] * 2.0 ** -22])
    e_grad = wt * (e_r + beta * e_em1 + 2.0 ** -22 * (free.abs() + beta * torch.expm1(x).abs()))
    return stats, e_stats, w, wt * grad, e_grad


def _run(wb, data, per_sequence, lo=0.2, hi=0.28, beta=0.1, dl=1.5):
    nll, old, ref, adv, labels = data
    kw = dict(ref_nll=ref, clip_low=lo, clip_high=hi, kl_weight=beta)
    stats, weight = wb.policy_loss(nll, old, adv, labels, per_sequence=per_sequence, **kw)
    dnll = wb.policy_loss_backward(torch.tensor(dl, device=DEV), nll, old, adv, labels, weight, **kw)
    assert wb.check_device_error() == 0
    return stats, weight, dnll


def _check(got, ref, labels, dl=1.5):
    (stats, weight, dnll), (want, e_stats, w, grad, e_grad) = got, ref
    assert bool(((stats.double() - want).abs() <= e_stats).all()), (stats.tolist(), want.tolist(), e_stats.tolist())
    assert bool(((weight.double() - w).abs() <= 2.0 ** -23 * w).all())
    assert not dnll[labels < 0].any()
    over = (dnll.double() - dl * grad).abs() - (dl * e_grad + 1e-36)
    assert float(over.max()) <= 0, float(over.max())


# up to 128 sequences of 512 tokens are one block's; a sequence has one to eight warps
SHAPES = [(1, 1), (1, 5), (3, 33), (128, 512), (128, 300), (129, 512), (40, 9), (8, 77), (5, 512), (5, 513), (9, 1025), (3, 2049), (2, 5000), (100, 448), (1300, 31), (10000, 7)]


@pytest.mark.parametrize("S,T", SHAPES)
@pytest.mark.parametrize("per_sequence", [False, True])
@pytest.mark.parametrize("per_token", [False, True])
def test_against_float64(wb, S, T, per_sequence, per_token):
    data = _data(S, T, S + T, per_token)
    _check(_run(wb, data, per_sequence), _reference(*data, 0.2, 0.28, 0.1, per_sequence), data[-1])


def _moved(t, elements):
    flat = torch.empty(t.numel() + elements, dtype=t.dtype, device=DEV)[elements:]
    return flat.copy_(t.reshape(-1)).view(t.shape)


# four tokens side by side where T is a multiple of 4 and every tensor lies on 16 bytes; one by one else
@pytest.mark.parametrize("S,T", [(200, 448), (131, 4), (300, 36), (7, 1028), (3, 4100), (2, 20000)])
@pytest.mark.parametrize("per_token,with_ref", [(False, True), (True, True), (False, False), (True, False)])
def test_tokens_on_and_off_16_bytes(wb, S, T, per_token, with_ref):
    data = _data(S, T, 2 * S + T, per_token)
    beta = 0.1 if with_ref else 0.0
    if not with_ref:
        data = data[:2] + (None,) + data[3:]
    want = _reference(*data, 0.2, 0.28, beta, False)
    first = _run(wb, data, False, beta=beta)
    _check(first, want, data[-1])
    for moved in range(5):
        off = tuple(_moved(t, 1) if i == moved and t is not None else t for i, t in enumerate(data))
        got = _run(wb, off, False, beta=beta)
        _check(got, want, data[-1])
        assert torch.equal(got[2], first[2])                    # a token's gradient does not depend on the path
    nll, old, ref, adv, labels = (None if t is None else t.clone() for t in data)
    for t in (nll, old) + ((ref,) if with_ref else ()) + ((adv,) if per_token else ()):
        t[labels < 0] = math.nan
    for a, b in zip(first, _run(wb, (nll, old, ref, adv, labels), False, beta=beta)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lo,hi,beta,with_ref", [(0.0, 0.0, 0.0, False), (1.0, 0.2, 0.0, True), (0.2, 1e30, 1.0, True), (0.1, 0.1, -0.3, True)])
def test_options(wb, lo, hi, beta, with_ref):
    nll, old, ref, adv, labels = _data(20, 100, 3)
    adv[4] = 0
    old[4] = nll[4] + 200                                       # an advantage of zero gives zero, whatever the ratio
    data = (nll, old, ref if with_ref else None, adv, labels)
    got = _run(wb, data, True, lo, hi, beta)
    ref64 = _reference(*data, lo, hi, beta, True)
    # a negative weight makes magnitudes of differences: the bound takes both parts as they are
    if beta < 0:
        ref64 = (ref64[0], _reference(*data, lo, hi, -beta, True)[1], ref64[2], ref64[3], _reference(*data, lo, hi, -beta, True)[4])
    _check(got, ref64, labels)


def test_values_that_take_no_part_reach_nothing(wb):
    data = _data(6, 70, 1)
    want = _run(wb, data, True)
    for bad in (math.nan, math.inf, -math.inf):
        nll, old, ref, adv, labels = (t.clone() for t in data)
        for t in (nll, old, ref):
            t[labels < 0] = bad
        adv[3] = bad                                             # the sequence without tokens
        for a, b in zip(want, _run(wb, (nll, old, ref, adv, labels), True)):
            assert torch.equal(a, b)
    nothing = (data[0], data[1], data[2], data[3], torch.full_like(data[4], -1))
    for x in _run(wb, nothing, False) + _run(wb, nothing, True):
        assert not x.any()


@pytest.mark.parametrize("S", [3, 400])
def test_losses_without_a_bound(wb, S):
    # a ratio beyond float32 under a negative advantage is not clipped: the loss is infinite, and so is that token's gradient, alone
    nll, old, ref, adv, labels = _data(S, 20, 2)
    labels[1, 3] = 7
    adv[:] = -1
    old[1, 3] = nll[1, 3] + 120
    stats, weight, dnll = _run(wb, (nll, old, None, adv, labels), False, beta=0.0, dl=1.0)
    assert float(stats[0]) == math.inf and math.isfinite(float(stats[2]))
    rest = dnll.clone()
    rest[1, 3] = 0
    assert float(dnll[1, 3]) == -math.inf and bool(torch.isfinite(rest).all())
    nll[1, 3] = math.nan
    assert math.isnan(float(_run(wb, (nll, old, None, adv, labels), True, beta=0.0)[0][0]))


def test_the_border_of_the_clip_is_decided_on_the_exact_difference(wb):
    # old - nll lies next to log1p(0.28) by less than a rounding of the difference
    t = math.log1p(0.28)
    S, T = 64, 400
    g = torch.Generator(device=DEV).manual_seed(9)
    nll = 4 + 8 * torch.rand(S, T, generator=g, device=DEV)
    old = (nll.double() + t).float()
    for i in range(T):                                           # steps of one float around it
        for _ in range(abs(i % 7 - 3)):
            old[:, i] = torch.nextafter(old[:, i], torch.full_like(old[:, i], math.inf if i % 7 > 3 else -math.inf))
    adv = torch.ones(S, device=DEV)
    labels = torch.zeros(S, T, dtype=torch.int64, device=DEV)
    stats, weight, dnll = _run(wb, (nll, old, None, adv, labels), False, beta=0.0)
    clipped = old.double() - nll.double() > t
    assert 0.2 < float(clipped.double().mean()) < 0.8
    assert torch.equal(dnll == 0, clipped)
    assert abs(float(stats[2]) - float(clipped.double().mean())) < 1e-6
    adv = -adv
    old = (nll.double() + math.log1p(-0.2)).float()
    stats, weight, dnll = _run(wb, (nll, old, None, adv, labels), False, beta=0.0)
    assert torch.equal(dnll == 0, old.double() - nll.double() < math.log1p(-0.2))


@pytest.mark.parametrize("x", [0.0, 1e-30, 1e-7, 1e-3, 0.1, 0.49, 0.51, -1e-4, -0.49, -0.51, -3.0, 20.0, -60.0])
def test_the_kl_term_over_its_range(wb, x):
    nll = torch.full((1, 3), 0.0, device=DEV)
    ref = torch.full((1, 3), -x, device=DEV)
    labels = torch.zeros(1, 3, dtype=torch.int64, device=DEV)
    stats, weight, dnll = _run(wb, (nll, nll.clone(), ref, torch.zeros(1, device=DEV), labels), False, beta=1.0, dl=1.0)
    xd = -ref[0, 0].double()
    # the series' and the difference's errors, the mean of three
    want = float(torch.expm1(xd) - xd) if abs(x) > 1e-4 else float(xd * xd / 2 * (1 + xd / 3 + xd * xd / 12))
    assert abs(float(stats[1]) - want) <= 2.0 ** -20 * want + 2.0 ** -149
    slope = float(torch.expm1(xd)) / 3
    assert bool(((dnll.double() - slope).abs() <= 2.0 ** -21 * abs(slope)).all())


@pytest.mark.parametrize("S,T", [(1, 1 << 20), (3, 700001), (1, 1 << 24)])
@pytest.mark.parametrize("d", [-0.15, 0.03, 0.11])
@pytest.mark.parametrize("per_token", [False, True])
def test_long_sequences(wb, S, T, d, per_token):
    # equal terms, whose roundings in one float32 would all go the same way.  32 at most are added in a row, the rest in pairs of float32
    # but for the last one of a lane (1), 32 lanes (5) and 8 warps (7): 2^-24 of the sum each
    nll, old, ref = (torch.full((S, T), c, device=DEV) for c in (1.0, 1.0 + d, 0.7))     # within a factor of 2: differences are exact
    adv = torch.full((S, T) if per_token else (S,), -1.0, device=DEV)
    labels = torch.zeros(S, T, dtype=torch.int64, device=DEV)
    labels[:, T - 5:] = -1
    ratio, x = math.exp(float(old[0, 0]) - 1.0), 1.0 - float(ref[0, 0])
    kl = math.expm1(x) - x
    for per_sequence in (False, True):
        stats, weight, dnll = _run(wb, (nll, old, ref, adv, labels), per_sequence)
        off = 2.0 ** -24 * (32 + 1 + 5 + 7) + 2.0 ** -22
        want = ratio + 0.1 * kl
        assert abs(float(stats[0]) - want) <= (off + 2.0 ** -20) * want
        assert abs(float(stats[1]) - kl) <= (off + 2.0 ** -20) * kl
        assert float(stats[2]) == 0
        w = 1 / (S * (T - 5))
        assert bool(((weight.double() - w).abs() <= 2.0 ** -23 * w).all())
        grad = 1.5 * w * (0.1 * math.expm1(x) - ratio)
        assert bool(((dnll[:, :T - 5].double() - grad).abs() <= 2.0 ** -19 * abs(grad)).all()) and not dnll[:, T - 5:].any()


@pytest.mark.parametrize("bad,want", [(math.inf, math.inf), (math.nan, math.nan)])
@pytest.mark.parametrize("at", [0, 3000, 9999, 20000])
def test_long_sequences_with_a_loss_that_is_not_finite(wb, bad, want, at):
    # what an infinite sum's roundings left is no number, and stays out of it; the sequence beside it is as it was
    nll, old, ref, adv, labels = _data(2, 20001, 8)
    labels[1, at], adv[:] = 7, -1
    old[1, at] = bad
    stats, weight, dnll = _run(wb, (nll, old, ref, adv, labels), True)
    assert math.isnan(float(stats[0])) if math.isnan(want) else float(stats[0]) == want
    assert math.isfinite(float(stats[1])) and math.isfinite(float(stats[2])) and bool(torch.isfinite(dnll[0]).all())


def test_gradient_against_differences(wb):
    nll, old, ref, adv, labels = _data(7, 60, 4)
    stats, weight, dnll = _run(wb, (nll, old, ref, adv, labels), True, dl=1.0)
    f = lambda z: _reference(z, old, ref, adv, labels, 0.2, 0.28, 0.1, True)[0][0]  # noqa: E731
    # steps of 1e-6, and no token within 1e-5 of a border of the clip
    d = old.double() - nll.double()
    near = (d - math.log1p(0.28)).abs().minimum((d - math.log1p(-0.2)).abs()) < 1e-5
    for i in range(0, 60, 7):
        step = torch.zeros_like(nll, dtype=torch.float64)
        step[:, i] = 1e-6
        if bool(near[:, i].any()):
            continue
        want = float(f(nll.double() + step) - f(nll.double() - step)) / 2e-6
        assert abs(float(dnll[:, i].double().sum()) - want) < 1e-8 + 1e-5 * float(dnll[:, i].abs().sum())


def test_same_bits_side_stream_captured_and_in_place(wb):
    data = _data(500, 200, 6)
    first = _run(wb, data, True)
    nll, old, ref, adv, labels = data
    kw = dict(ref_nll=ref, clip_low=0.2, clip_high=0.28, kl_weight=0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stats, weight = wb.policy_loss(nll, old, adv, labels, per_sequence=True, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(stats, first[0]) and torch.equal(weight, first[1])
    dl = torch.tensor(1.5, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stats, weight = wb.policy_loss(nll, old, adv, labels, per_sequence=True, **kw)
        dnll = wb.policy_loss_backward(dl, nll, old, adv, labels, weight, **kw)
    for _ in range(2):
        for t in (stats, weight, dnll):
            t.fill_(3)
        graph.replay()
    for a, b in zip(first, (stats, weight, dnll)):
        assert torch.equal(a, b)


def test_python_refusals(wb):
    nll, old, ref, adv, labels = _data(4, 9, 1)
    for bad in (lambda: wb.policy_loss(nll, old, adv, labels, kl_weight=0.1), lambda: wb.policy_loss(nll.half(), old, adv, labels),
                lambda: wb.policy_loss(nll, old[:2], adv, labels), lambda: wb.policy_loss(nll, old, adv[:2], labels),
                lambda: wb.policy_loss(nll, old, adv, labels.int()), lambda: wb.policy_loss(nll.T, old.T, adv, labels.T),
                lambda: wb.policy_loss_backward(1.0, nll, old, adv, labels, adv), lambda: wb.policy_loss_backward(adv, nll, old, adv, labels, adv),
                lambda: wb.policy_loss_backward(adv[:1], nll, old, adv, labels, adv[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(wb.WbError):
        wb.policy_loss(nll, old, adv, labels, clip_low=1.5)
