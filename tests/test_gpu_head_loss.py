"""Vocabulary losses from hidden states and projection matrix (GPU) against float64 evaluations.

How far a result may be off is computed beside it.  A logit is a sum of d exact products in fp32: it
may be off by es = 2^-18 sum |x w| (64 roundings of the sum's magnitude).  A loss then is off by 2 es
(its logit and the lse) and the fp32 roundings of its terms.  D = softmax - target is off by
q (expm1 of 2 es and 2^-20) and rounded to bf16 (half a step, 2^-8); a gradient sums |D| |factor| of
those, is off by 2^-18 of that sum's magnitude again, and is rounded to bf16 (2^-8)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = 2.0 ** -8


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _data(M, d, V, seed, spread=1.0):
    g = _gen(seed)
    x = torch.randn(M, d, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(V, d, generator=g, device=DEV) * (spread / math.sqrt(d))).to(torch.bfloat16)
    dloss = (0.5 + torch.rand(M, generator=g, device=DEV)) / max(M, 1)
    return x, w, dloss, g


def _reference(x, w, target, valid, dloss, T):
    """target float64 [M, V]; returns values and how far they may be off."""
    xd = torch.where(valid[:, None], x.double(), 0.0)
    wd = w.double()
    s = xd @ wd.T / T
    mag = xd.abs() @ wd.abs().T / T
    es = 2.0 ** -18 * mag.amax(1)
    lse = torch.logsumexp(s, 1)
    q = torch.exp(s - lse[:, None])
    kl = T * T * (torch.special.xlogy(target, target) - target * (s - lse[:, None]))
    loss = kl.sum(1)
    parts = T * T * (torch.special.xlogy(target, target).abs() + target * (s.abs() + lse[:, None].abs()))
    e_loss = T * T * 2 * es + 2.0 ** -20 * parts.sum(1) + 2.0 ** -20
    e_lse = es + 2.0 ** -21 * (lse.abs() + s.abs().amax(1) + 1)
    D = torch.where(valid[:, None], q - target, 0.0)
    eD = torch.where(valid[:, None], HALF * D.abs() * 1.01 + q * torch.expm1(2 * es + 2.0 ** -20)[:, None] + 2.0 ** -22 * target, 0.0)
    f = torch.where(valid, dloss.double() * T, 0.0)[:, None]
    dx = (f * D) @ wd
    e_dx = (f.abs() * (eD + 2.0 ** -18 * D.abs())) @ wd.abs() + HALF * dx.abs() * 1.01 + 1e-30
    dw = (f * D).T @ xd
    # x dloss / max|dloss| is rounded to bf16 too
    e_dw = (f.abs() * (eD + (2.0 ** -18 + HALF) * D.abs())).T @ xd.abs() * 1.01 + HALF * dw.abs() * 1.01 + 1e-30
    zero = torch.zeros_like(loss)
    return {"loss": (torch.where(valid, loss, zero), e_loss), "lse": (torch.where(valid, lse, zero), e_lse), "dx": (dx, e_dx), "dw": (dw, e_dw)}


def _check(got, ref, names):
    for name in names:
        value, off = ref[name]
        g = got[name].double()
        assert g.shape == value.shape and torch.isfinite(g).all(), name
        over = ((g - value).abs() - off).max()
        assert float(over) <= 0, (name, float(over), float(((g - value).abs() / off).max()))


def _ce(wb, x, w, labels, dloss, smooth):
    loss, lse = wb.linear_cross_entropy(x, w, labels, smooth)
    dx, dw = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, smooth)
    assert wb.check_device_error() == 0
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def _ce_target(labels, V, smooth):
    t = torch.full((labels.numel(), V), smooth / V, device=DEV, dtype=torch.float64)
    return t.scatter_add_(1, labels.clamp(min=0)[:, None], torch.full((labels.numel(), 1), 1 - smooth, device=DEV, dtype=torch.float64))


CE = [(1, 8, 1), (1, 64, 2), (3, 8, 5), (1, 1280, 5003), (5, 72, 255), (128, 64, 256), (129, 136, 257), (77, 384, 1000),
      (300, 384, 2049), (1000, 256, 513), (257, 1280, 3001), (64, 2056, 700), (8, 40, 333), (16, 1288, 700), (2, 4104, 300), (17, 768, 900),
      (450, 768, 1100), (2, 4096, 5000)]


@pytest.mark.parametrize("M,d,V", CE)
@pytest.mark.parametrize("smooth", [0.0, 0.1])
@pytest.mark.parametrize("holes", [False, True])
def test_cross_entropy_matches_the_formulas(wb, M, d, V, smooth, holes):
    x, w, dloss, g = _data(M, d, V, M + d + V, spread=2.0)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    if holes:
        labels[torch.rand(M, generator=g, device=DEV) < 0.4] = -100
    valid = labels >= 0
    ref = _reference(x, w, _ce_target(labels, V, smooth), valid, dloss, 1.0)
    # the target's entropy is not part of a cross entropy
    t = _ce_target(labels, V, smooth)
    ref["loss"] = (torch.where(valid, ref["loss"][0] - torch.special.xlogy(t, t).sum(1), 0.0), ref["loss"][1])
    _check(_ce(wb, x, w, labels, dloss, smooth), ref, ("loss", "lse", "dx", "dw"))


def _distill_target(top, index, V, T):
    there = (index >= 0) & (top.double() > -math.inf)
    valid = there.any(1)
    t = torch.where(there, top.double() / T, -math.inf)
    p = torch.where(valid[:, None], torch.exp(t - torch.where(valid, t.amax(1), 0.0)[:, None]), 0.0)
    p = p / torch.where(valid, p.sum(1), 1.0)[:, None]
    return torch.zeros(index.shape[0], V, device=DEV, dtype=torch.float64).scatter_add_(1, index.clamp(min=0), p), valid


def _distill(wb, x, w, top, index, dloss, T):
    loss, lse = wb.linear_distill(x, w, top, index, T)
    dx, dw = wb.linear_distill_backward(dloss, x, w, top, index, lse, T)
    assert wb.check_device_error() == 0
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


DISTILL = [(1, 8, 1, 1), (2, 64, 7, 3), (1, 384, 5003, 100), (130, 72, 300, 16), (257, 384, 1027, 64), (65, 128, 2000, 1),
           (9, 64, 3001, 1024), (513, 256, 777, 9)]


@pytest.mark.parametrize("M,d,V,k", DISTILL)
@pytest.mark.parametrize("T", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_distillation_matches_the_formulas(wb, M, d, V, k, T, kind):
    x, w, dloss, g = _data(M, d, V, M + d + V + k)
    index = torch.randint(0, V, (M, k), generator=g, device=DEV)       # the same index twice is common here
    index[torch.rand(M, k, generator=g, device=DEV) < 0.2] = -1
    top = (3 * torch.randn(M, k, generator=g, device=DEV)).to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[kind])
    top[torch.rand(M, k, generator=g, device=DEV) < 0.1] = -math.inf
    if M > 4:
        index[3] = -1                                                   # rows without any entry
        top[4] = -math.inf
    target, valid = _distill_target(top, index, V, T)
    _check(_distill(wb, x, w, top, index, dloss, T), _reference(x, w, target, valid, dloss, T), ("loss", "lse", "dx", "dw"))


def test_several_pieces_of_the_vocabulary(wb):
    # rows enough that the backward pass takes the vocabulary in pieces, the last one ragged
    M, d, V = 9000, 64, 30011
    x, w, dloss, g = _data(M, d, V, 17, spread=3.0)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    labels[::7] = -1
    got = _ce(wb, x, w, labels, dloss, 0.0)
    want = {n: torch.zeros(s, device=DEV, dtype=torch.float64) for n, s in (("loss", M), ("dx", (M, d)), ("dw", (V, d)))}
    for i in range(0, M, 1500):
        j = slice(i, i + 1500)
        xd = torch.where((labels[j] >= 0)[:, None], x[j].double(), 0.0)
        lq = torch.log_softmax(xd @ w.double().T, 1)
        lab = labels[j].clamp(min=0)
        want["loss"][j] = torch.where(labels[j] >= 0, -lq.gather(1, lab[:, None])[:, 0], 0.0)
        D = lq.exp()
        D.scatter_add_(1, lab[:, None], torch.full_like(D[:, :1], -1.0))
        D *= torch.where(labels[j] >= 0, dloss[j].double(), 0.0)[:, None]
        want["dx"][j] = D @ w.double()
        want["dw"] += D.T @ xd
    # three roundings to bf16 of rms 2^-8 / sqrt(3) each: 2-norms within 2^-8
    for name, tol in (("loss", 1e-6), ("dx", HALF), ("dw", HALF)):
        rel = float((got[name].double() - want[name]).norm() / want[name].norm())
        assert rel < tol, (name, rel)
    assert not got["dx"][::7].any() and not got["loss"][::7].any()


def test_rows_that_take_no_part_reach_nothing(wb):
    M, d, V = 333, 128, 901
    x, w, dloss, g = _data(M, d, V, 3)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    out = torch.rand(M, generator=g, device=DEV) < 0.5
    labels[out] = -100
    clean = _ce(wb, x, w, labels, dloss, 0.0)
    dirty_x, dirty_d = x.clone(), dloss.clone()
    dirty_x[out] = float("nan")
    dirty_d[out] = float("inf")
    dirty = _ce(wb, dirty_x, w, labels, dirty_d, 0.0)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n


@pytest.mark.parametrize("M", [1, 200])
def test_no_row_takes_part(wb, M):
    x, w, dloss, _ = _data(M, 64, 300, 4)
    x[:] = float("nan")
    got = _ce(wb, x, w, torch.full((M,), -1, device=DEV), dloss, 0.1)
    for n in got:
        assert not got[n].any(), n
    got = _distill(wb, x, w, torch.zeros(M, 2, device=DEV), torch.full((M, 2), -1, device=DEV), dloss, 2.0)
    for n in got:
        assert not got[n].any(), n


def test_no_rows(wb):
    x, w, dloss, _ = _data(0, 64, 300, 4)
    got = _ce(wb, x, w, torch.zeros(0, dtype=torch.int64, device=DEV), dloss, 0.0)
    assert got["loss"].shape == (0,) and got["dx"].shape == (0, 64) and not got["dw"].any()


@pytest.mark.parametrize("M", [12, 40, 300])
def test_a_target_past_the_vocabulary_is_a_loss_of_nan(wb, M):
    d, V = 64, 100
    x, w, dloss, g = _data(M, d, V, 8)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    without = labels.clone()
    without[5] = -1
    labels[5] = V
    got, ref = _ce(wb, x, w, labels, dloss, 0.0), _ce(wb, x, w, without, dloss, 0.0)
    assert torch.isnan(got["loss"][5]) and int(torch.isnan(got["loss"]).sum()) == 1
    for n in ("lse", "dx", "dw"):
        assert torch.equal(got[n], ref[n])
    assert got["lse"][5] == 0
    index = torch.randint(0, V, (M, 4), generator=g, device=DEV)
    index[7, 2] = V + 3
    got = _distill(wb, x, w, torch.randn(M, 4, device=DEV), index, dloss, 1.0)
    assert torch.isnan(got["loss"][7]) and int(torch.isnan(got["loss"]).sum()) == 1
    assert not got["dx"][7].any() and torch.isfinite(got["dw"].float()).all()


@pytest.mark.parametrize("M", [6, 60, 400])
def test_teacher_values_of_absent_entries_do_not_matter(wb, M):
    d, V, k = 64, 700, 9
    x, w, dloss, g = _data(M, d, V, 14)
    index = torch.randint(0, V, (M, k), generator=g, device=DEV)
    top = torch.randn(M, k, generator=g, device=DEV)
    gone = torch.rand(M, k, generator=g, device=DEV) < 0.4
    index[gone] = -5
    clean = _distill(wb, x, w, top, index, dloss, 1.5)
    dirty = top.clone()
    dirty[gone] = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).repeat(M * k)[:int(gone.sum())]
    for n, v in _distill(wb, x, w, dirty, index, dloss, 1.5).items():
        assert torch.equal(v, clean[n]), n


def test_not_a_number_stays_in_its_row(wb):
    for M in (7, 50, 400):
        x, w, dloss, g = _data(M, 64, 700, 15)
        labels = torch.randint(0, 700, (M,), generator=g, device=DEV)
        clean = _ce(wb, x, w, labels, dloss, 0.0)
        x[3, 5] = float("nan")
        got = _ce(wb, x, w, labels, dloss, 0.0)
        for n in ("loss", "lse", "dx"):
            bad = torch.isnan(got[n]).reshape(M, -1)
            assert bad[3].all() and int(bad.any(1).sum()) == 1
            keep = torch.arange(M, device=DEV) != 3
            assert torch.equal(got[n][keep], clean[n][keep])


def test_extreme_logits(wb):
    # one column takes everything, and logits of thousands: no overflow, loss 0 or the difference
    M, d, V = 130, 64, 1000
    x = torch.zeros(M, d, device=DEV, dtype=torch.bfloat16)
    w = torch.zeros(V, d, device=DEV, dtype=torch.bfloat16)
    x[:, 0] = 64
    w[:, 0] = torch.linspace(-100, 100, V, device=DEV).to(torch.bfloat16)
    w[777, 0] = 200
    labels = torch.full((M,), 777, device=DEV)
    labels[1::2] = 3
    loss, lse = wb.linear_cross_entropy(x, w, labels)
    s = 64 * w[:, 0].double()
    torch.testing.assert_close(lse.double(), torch.full((M,), float(s[777]), device=DEV, dtype=torch.float64), rtol=2 ** -21, atol=0)
    torch.testing.assert_close(loss[::2], torch.zeros_like(loss[::2]), rtol=0, atol=2e-3)
    torch.testing.assert_close(loss[1::2].double(), torch.full_like(loss[1::2], float(s[777] - s[3])).double(), rtol=2 ** -21, atol=2e-3)


def test_cross_entropy_is_distillation_from_one_certain_entry(wb):
    M, d, V = 200, 320, 1501
    x, w, dloss, g = _data(M, d, V, 12)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    a = _ce(wb, x, w, labels, dloss, 0.0)
    b = _distill(wb, x, w, torch.full((M, 1), 7.0, device=DEV), labels[:, None].contiguous(), dloss, 1.0)
    torch.testing.assert_close(a["loss"], b["loss"], rtol=2 ** -20, atol=2 ** -20)
    for n in ("lse", "dx", "dw"):
        assert torch.equal(a[n], b[n]), n


def test_gradients_match_differences(wb):
    # directional derivative of sum dloss loss along a direction of x and w, on inputs whose steps are
    # exact in bf16: x and w on a grid of 2^-4, moved by 2^-6
    M, d, V, k, T = 40, 32, 77, 5, 2.0
    g = _gen(23)
    x = (torch.randint(-16, 17, (M, d), generator=g, device=DEV) / 16).to(torch.bfloat16)
    w = (torch.randint(-16, 17, (V, d), generator=g, device=DEV) / 16).to(torch.bfloat16)
    vx = torch.randint(-1, 2, (M, d), generator=g, device=DEV).float()
    vw = torch.randint(-1, 2, (V, d), generator=g, device=DEV).float()
    dloss = torch.rand(M, generator=g, device=DEV)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    index = torch.randint(0, V, (M, k), generator=g, device=DEV)
    top = torch.randn(M, k, generator=g, device=DEV)
    h = 2.0 ** -6

    for forward, backward in ((lambda a, b: wb.linear_cross_entropy(a, b, labels, 0.1),
                               lambda lse: wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, 0.1)),
                              (lambda a, b: wb.linear_distill(a, b, top, index, T),
                               lambda lse: wb.linear_distill_backward(dloss, x, w, top, index, lse, T))):
        def value(e):
            a, b = (x.float() + e * vx).to(torch.bfloat16), (w.float() + e * vw).to(torch.bfloat16)
            assert torch.equal(a.float(), x.float() + e * vx) and torch.equal(b.float(), w.float() + e * vw)
            return float((forward(a, b)[0].double() * dloss).sum())

        dx, dw = backward(forward(x, w)[1])
        want = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
        # fourth-order difference: its error is h^4 / 30 of the fifth derivative
        slope = (8 * (value(h) - value(-h)) - (value(2 * h) - value(-2 * h))) / (12 * h)
        # gradients rounded to bf16 twice over: 2^-7 of the terms' magnitude over sqrt of their number, times 4
        terms = torch.cat([(dx.double() * vx).flatten(), (dw.double() * vw).flatten()])
        assert abs(slope - want) < 4 * 2.0 ** -7 * float(terms.norm()) + 1e-3 * abs(want), (slope, want)


def test_gradients_that_are_not_wanted(wb):
    M, d, V = 70, 64, 500
    x, w, dloss, g = _data(M, d, V, 2)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    _, lse = wb.linear_cross_entropy(x, w, labels)
    dx, dw = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse)
    a, none = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, need_dw=False)
    assert none is None and torch.equal(a, dx)
    none, b = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, need_dx=False)
    assert none is None and torch.equal(b, dw)


def test_same_bits_every_time_on_a_side_stream_and_in_a_graph(wb):
    M, d, V, k = 400, 384, 3000, 12
    x, w, dloss, g = _data(M, d, V, 31)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    labels[::5] = -1
    index = torch.randint(0, V, (M, k), generator=g, device=DEV)
    top = torch.randn(M, k, generator=g, device=DEV)

    def both(stream=None):
        loss, lse = wb.linear_cross_entropy(x, w, labels, 0.1, stream=stream)
        dx, dw = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse, 0.1, stream=stream)
        kl, lse2 = wb.linear_distill(x, w, top, index, 2.0, stream=stream)
        return (loss, lse, dx, dw, kl, lse2, *wb.linear_distill_backward(dloss, x, w, top, index, lse2, 2.0, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    labels.copy_(labels.roll(1))
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(both(), got):
        assert torch.equal(a, b)
    assert wb.check_device_error() == 0


def test_a_training_step_of_a_head(wb):
    # the operators together: final norm, projection and loss, and the way back, two losses added
    B, T, d, V, k = 3, 45, 384, 1200, 8
    g = _gen(77)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    h, res = n(B, T, d).to(torch.bfloat16), n(B, T, d).to(torch.bfloat16)
    gamma, beta = 1 + 0.1 * n(d), 0.1 * n(d)
    w = (n(V, d) * 0.1).to(torch.bfloat16)
    labels = torch.randint(0, V, (B, T), generator=g, device=DEV)
    for b, length in enumerate((45, 20, 1)):
        labels[b, length:] = -100
    index = torch.randint(0, V, (B * T, k), generator=g, device=DEV)
    index[labels.flatten() < 0] = -1
    top = n(B * T, k)
    valid = labels.flatten() >= 0
    dloss = torch.full((B * T,), 1.0 / int(valid.sum()), device=DEV)

    y, total, stats = wb.layernorm_forward(h, gamma, beta, residual=res)
    y2 = y.view(B * T, d)
    ce, lse1 = wb.linear_cross_entropy(y2, w, labels.flatten())
    kl, lse2 = wb.linear_distill(y2, w, top, index, 2.0)
    dx1, dw1 = wb.linear_cross_entropy_backward(dloss, y2, w, labels.flatten(), lse1)
    dx2, dw2 = wb.linear_distill_backward(dloss, y2, w, top, index, lse2, 2.0)
    dy = (dx1.float() + dx2.float()).to(torch.bfloat16).view(B, T, d)
    dh, dgamma, dbeta = wb.layernorm_backward(dy, total, gamma, stats)
    assert wb.check_device_error() == 0

    # the same in float64 by automatic differentiation, from the stored (rounded) sum
    t64, g64, b64, w64 = (a.double().requires_grad_() for a in (total, gamma, beta, w))
    y64 = torch.nn.functional.layer_norm(t64, (d,), g64, b64, 1e-5).view(B * T, d)
    s = y64 @ w64.T
    target, _ = _distill_target(top, index, V, 2.0)
    l1 = torch.nn.functional.cross_entropy(s, labels.flatten(), ignore_index=-100, reduction="sum")
    l2 = (4 * (torch.special.xlogy(target, target) - target * torch.log_softmax(s / 2, 1)).sum(1))[valid].sum()
    loss64 = (l1 + l2) / int(valid.sum())
    loss64.backward()
    loss64 = float(loss64.detach())
    # y is rounded to bf16 (2^-8) on its way into the logits; the loss moves by its gradient times that
    got = float(((ce + kl) * dloss).double().sum())
    assert abs(got - loss64) < 2.0 ** -8 * loss64
    # a gradient goes through at most six roundings to bf16 here (y, D, x', dx, their sum, dh), rms 2^-8 / sqrt(3) each
    tol = 6 ** 0.5 * 2.0 ** -8
    for name, a, b in (("dh", dh, t64.grad), ("dw", dw1.double() + dw2.double(), w64.grad), ("dgamma", dgamma, g64.grad), ("dbeta", dbeta, b64.grad)):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < tol, (name, rel)
    assert not dh[1, 20:].any() and not dh[2, 1:].any()


def test_refusals(wb):
    M, d, V = 8, 64, 100
    x, w, dloss, g = _data(M, d, V, 1)
    labels = torch.zeros(M, dtype=torch.int64, device=DEV)
    top, index = torch.zeros(M, 3, device=DEV), torch.zeros(M, 3, dtype=torch.int64, device=DEV)
    lse = torch.zeros(M, device=DEV)
    for bad in (lambda: wb.linear_cross_entropy(x.float(), w, labels),
                lambda: wb.linear_cross_entropy(x, w.half(), labels),
                lambda: wb.linear_cross_entropy(x, w[:, :32].contiguous(), labels),
                lambda: wb.linear_cross_entropy(x, w, labels.int()),
                lambda: wb.linear_cross_entropy(x, w, labels[:4]),
                lambda: wb.linear_cross_entropy(x.view(2, 4, d), w, labels),
                lambda: wb.linear_cross_entropy(x.t(), w, labels),
                lambda: wb.linear_cross_entropy_backward(dloss[:4], x, w, labels, lse),
                lambda: wb.linear_cross_entropy_backward(dloss.double(), x, w, labels, lse),
                lambda: wb.linear_distill(x, w, top.double(), index),
                lambda: wb.linear_distill(x, w, top[:, 0].contiguous(), index),
                lambda: wb.linear_distill(x, w, top, index[:, :2].contiguous()),
                lambda: wb.linear_distill(x, w, top, index.int())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wb.linear_cross_entropy(x, w, labels, 1.0),
                lambda: wb.linear_cross_entropy(x, w, labels, -0.1),
                lambda: wb.linear_cross_entropy(x, w, labels, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
                lambda: wb.linear_cross_entropy(x[:, :60].contiguous(), w[:, :60].contiguous(), labels),
                lambda: wb.linear_distill(x, w, top, index, 0.0),
                lambda: wb.linear_distill(x, w, top, index, float("inf")),
                lambda: wb.linear_distill(x, w, top[:, :0].contiguous(), index[:, :0].contiguous())):
        with pytest.raises(wb.WbError):
            bad()
