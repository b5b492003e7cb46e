"""The training operators where values are at their edges (GPU), against float64 evaluations."""
import pytest
import torch

from test_gpu_head_loss import _check, _data, _distill, _distill_target, _reference

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
