"""The training operators where values are at their edges (GPU), against float64 evaluations."""
import math

import pytest
import torch

from test_gpu_head_loss import _ce, _check, _data, _distill, _distill_target, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("tops", [1, 2, 10, 100])
@pytest.mark.parametrize("T", [1.0, 0.5])
@pytest.mark.parametrize("M", [12, 161])
def test_teacher_logits_far_below_the_top(wb, tops, T, M):
    # exp of such a gap is subnormal in float32 or zero, and so is its share of the row's sum; no value that
    # enters the float64 reference is: its share is below 2^-140, nothing against the bounds
    d, V = 64, 1500
    x, w, dloss, g = _data(M, d, V, M + tops)
    gaps = torch.linspace(101.4, 104.2, M, device=DEV) if M == 12 else torch.linspace(95, 105, M, device=DEV)
    top = torch.full((M, tops + 3), 7.0, device=DEV)
    top[:, -3:] -= gaps[:, None] * torch.tensor([1.0, 1.0, 0.995], device=DEV)
    index = torch.stack([torch.randperm(V, generator=g, device=DEV)[:tops + 3] for _ in range(M)])
    index[1::2, -2] = index[1::2, -3]                              # the same entry twice, both far below
    top = (top * T).contiguous()
    target, valid = _distill_target(top, index, V, T)
    assert bool(valid.all())
    _check(_distill(wb, x, w, top, index, dloss, T), _reference(x, w, target, valid, dloss, T), ("loss", "lse", "dx", "dw"))


@pytest.mark.parametrize("low", [-1e10, -1e30, -1.5e38, torch.finfo(torch.bfloat16).min, -math.inf])
@pytest.mark.parametrize("M", [4, 60, 300])
def test_vocabulary_entries_masked_by_a_low_logit(wb, low, M):
    # one feature lowers 300 entries in a row (whole tiles' shares of columns among them): they take no part at all,
    # so everything is as over the other entries alone
    d, V, lo, hi = 64, 1000, 100, 400
    x, w, dloss, g = _data(M, d, V, 43)
    x[:, 0] = 1
    w[:, 0] = 0
    w[lo:hi, 0] = low
    keep = torch.ones(V, dtype=torch.bool, device=DEV)
    keep[lo:hi] = False
    label = torch.randint(0, V - (hi - lo), (M,), generator=g, device=DEV)
    target = torch.zeros(M, int(keep.sum()), dtype=torch.float64, device=DEV).scatter_(1, label[:, None], 1.0)
    labels = torch.where(label < lo, label, label + (hi - lo))
    ref = _reference(x, w[keep], target, torch.ones(M, dtype=torch.bool, device=DEV), dloss, 1.0)
    loss, lse = wb.linear_cross_entropy(x, w, labels)
    _check({"loss": loss, "lse": lse}, ref, ("loss", "lse"))
    kl, lse2 = wb.linear_distill(x, w, torch.zeros(M, 1, device=DEV), labels[:, None].contiguous())
    _check({"loss": kl, "lse": lse2}, ref, ("loss", "lse"))
    dx, dw = wb.linear_cross_entropy_backward(dloss, x, w, labels, lse)
    assert wb.check_device_error() == 0
    assert not dw[lo:hi].any()
    if low == -math.inf:              # 0 * -infinity, in the lowered feature alone
        assert torch.isnan(dx[:, 0]).all()
        dx[:, 0] = ref["dx"][0][:, 0].to(torch.bfloat16)
    _check({"dx": dx, "dw": dw[keep]}, ref, ("dx", "dw"))


@pytest.mark.parametrize("T", [1e-30, 1e-20, 1e-3, 7.0])
@pytest.mark.parametrize("M", [5, 70])
def test_the_loss_at_small_and_large_temperatures(wb, T, M):
    # one certain entry: the loss is T (T lse - s), its parts far outside of float32's range of squares.  Logits and
    # lse are off as in test_gpu_head_loss, relative to themselves; the factor T^2 has two roundings more
    d, V = 64, 300
    x, w, _, g = _data(M, d, V, 41)
    label = torch.randint(0, V, (M, 1), generator=g, device=DEV)
    loss, lse = wb.linear_distill(x, w, torch.full((M, 1), 1e10, device=DEV), label, T)
    assert wb.check_device_error() == 0
    f = torch.tensor(T, dtype=torch.float32).double().item()
    s = x.double() @ w.double().T / f
    want = torch.logsumexp(s, 1)
    mag = (x.double().abs() @ w.double().abs().T).amax(1) / f
    e_lse = 2.0 ** -18 * mag + 2.0 ** -21 * (want.abs() + 1)
    assert bool(((lse.double() - want).abs() <= e_lse).all())
    kl = (want - s.gather(1, label)[:, 0])
    assert bool(((loss.double() - f * f * kl).abs() <= f * f * (2 * e_lse + 2.0 ** -22 * kl.abs())).all())


@pytest.mark.parametrize("T", [1e-30, 1e-20, 1e-10])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_gradients_at_small_temperatures(wb, T, M):
    # logits on a grid of 2^-8, exact in every form of the product; over such a T each step of the grid is at least
    # 2^25, so the softmax is all at the largest logit.  D is then -1, 0 or 1, and only the results are rounded
    d, V = 64, 300
    g = torch.Generator(device=DEV).manual_seed(M)
    x = (torch.randint(-16, 17, (M, d), generator=g, device=DEV) / 16).to(torch.bfloat16)
    w = (torch.randint(-16, 17, (V, d), generator=g, device=DEV) / 16).to(torch.bfloat16)
    s = x.double() @ w.double().T
    most, first = s.max(1)
    valid = (s == most[:, None]).sum(1) == 1                      # no softmax to compare with where two are the largest
    label = torch.randint(0, V, (M,), generator=g, device=DEV)
    label[::3] = first[::3]                                       # rows whose softmax is their target
    index = torch.where(valid, label, -1)[:, None].contiguous()
    dloss = torch.full((M,), 0.25, device=DEV)
    top = torch.zeros(M, 1, device=DEV)
    _, lse = wb.linear_distill(x, w, top, index, T)
    dx, dw = wb.linear_distill_backward(dloss, x, w, top, index, lse, T)
    assert wb.check_device_error() == 0 and int(valid.sum()) > M // 2
    D = torch.zeros(M, V, dtype=torch.float64, device=DEV)
    D[torch.arange(M, device=DEV), first] += 1
    D[torch.arange(M, device=DEV), label] -= 1
    D *= torch.where(valid, 0.25 * torch.tensor(T, dtype=torch.float32).double().item(), 0.0)[:, None]
    # sums of such terms are exact in float32; the scale and the result are rounded, 2^-24 each and 2^-8
    for got, want in ((dx, D @ w.double()), (dw, D.T @ x.double())):
        assert bool(((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.abs()).all())


def test_more_rows_than_a_thousand_blocks_of_the_row_map_take_at_once(wb):
    M, d, V = 700_003, 8, 5
    x, w, dloss, g = _data(M, d, V, 44)
    labels = torch.randint(-1, V, (M,), generator=g, device=DEV)
    valid = labels >= 0
    target = torch.zeros(M, V, dtype=torch.float64, device=DEV).scatter_(1, labels.clamp(min=0)[:, None], 1.0)
    ref = _reference(x, w, target, valid, dloss, 1.0)
    _check(_ce(wb, x, w, labels, dloss, 0.0), ref, ("loss", "lse", "dx", "dw"))


def test_statistics_on_8_bytes(wb):
    # a slice of the statistics of a larger batch
    x = torch.randn(65, 384, device=DEV).to(torch.bfloat16)
    dy = torch.randn_like(x)
    gamma = torch.rand(384, device=DEV)
    _, _, stats = wb.layernorm_forward(x, gamma, gamma)
    part = wb.layernorm_backward(dy[1:], x[1:], gamma, stats[1:])
    whole = wb.layernorm_backward(dy[1:], x[1:], gamma, stats[1:].clone())
    for a, b in zip(part, whole):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M", [4, 60, 300])
def test_infinite_logits(wb, M):
    # w's first column is -infinity for 300 entries (a whole tile of columns and more): where x's first is 1 their
    # logits are -infinity and take no part; where it is -1 they are +infinity and the row has no softmax
    d, V = 64, 1000
    x, w, _, g = _data(M, d, V, 43)
    x[:, 0] = 1
    w[:300, 0] = -float("inf")
    labels = torch.randint(300, V, (M,), generator=g, device=DEV)
    loss, lse = wb.linear_cross_entropy(x, w, labels)
    s = x.double() @ w.double().T
    want = torch.logsumexp(s, 1)
    tol = 2.0 ** -18 * (x.double().abs() @ w[300:].double().abs().T).amax(1) + 2.0 ** -21 * (want.abs() + 8)
    assert bool(((lse.double() - want).abs() <= tol).all())
    assert bool(((loss.double() - (want - s.gather(1, labels[:, None])[:, 0])).abs() <= 2 * tol).all())
    # a target among them is infinitely unlikely, and so is smoothing over them
    gone = labels.clone()
    gone[1] = 7
    assert wb.linear_cross_entropy(x, w, gone)[0][1] == float("inf")
    assert torch.isfinite(wb.linear_cross_entropy(x, w, gone)[0]).sum() == M - 1
    assert bool((wb.linear_cross_entropy(x, w, labels, 0.1)[0] == float("inf")).all())
    kl, lse_t = wb.linear_distill(x, w, torch.zeros(M, 1, device=DEV), gone[:, None].contiguous())
    assert kl[1] == float("inf") and torch.isfinite(kl).sum() == M - 1 and torch.equal(lse_t, lse)
    x[2, 0] = -1
    bad, _ = wb.linear_cross_entropy(x, w, labels)
    assert not torch.isfinite(bad[2]) and torch.isfinite(bad).sum() == M - 1
    assert torch.equal(bad[3:], loss[3:]) and torch.equal(bad[:2], loss[:2])
    assert wb.check_device_error() == 0


def test_an_index_past_the_vocabulary_is_a_mistake_beside_any_logit(wb):
    x, w, _, _ = _data(20, 64, 50, 45)
    index = torch.arange(40, device=DEV).view(20, 2) % 50
    index[3, 1] = 50
    top = torch.zeros(20, 2, device=DEV)
    top[:, 1] = -math.inf
    loss, lse = wb.linear_distill(x, w, top, index)
    assert torch.isnan(loss[3]) and lse[3] == 0 and int(torch.isnan(loss).sum()) == 1
