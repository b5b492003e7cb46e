"""LayerNorm for training (GPU): dg and db of the backward pass over many rows, where every team of a block adds
several rows, its ring fills again, and the teams and blocks are joined; the forward pass of ragged rows on both
sides of the widths where its form changes.

The reference of the sums takes the call's own float32 statistics, so only the sums are in question.  A sum of n terms in
any order, at most `adds` additions in a row, is off by adds 2^-24 of the sum of magnitudes; a block adds
ceil(rows / 152) rows at most one after the other, then its teams (16 at most), then the partial rows in 32
slices of 5 and the slices.  A term dy (x - mean) rstd has two roundings more, and one where it is added."""
import pytest
import torch

from test_gpu_layernorm_train import _close, _inputs, _reference

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _adds(rows):
    return (rows + 151) // 152 + 16 + 5 + 32


def _check(dg, db, x, stats, dy, rows):
    want_g, want_b, mag_g, mag_b = (torch.zeros(x.shape[1], dtype=torch.float64, device=DEV) for _ in range(4))
    for i in range(0, x.shape[0], 1 << 12):
        j = slice(i, i + (1 << 12))
        h = (x[j].double() - stats[j, :1].double()) * stats[j, 1:].double()
        y = dy[j].double()
        want_g += (y * h).sum(0)
        want_b += y.sum(0)
        mag_g += (y * h).abs().sum(0)
        mag_b += y.abs().sum(0)
    unit = 2.0 ** -24 * 1.01
    over_g = ((dg.double() - want_g).abs() - unit * (_adds(rows) + 3) * mag_g).max()
    over_b = ((db.double() - want_b).abs() - unit * _adds(rows) * mag_b).max()
    assert float(over_g) <= 0 and float(over_b) <= 0, (float(over_g), float(over_b))


# widths of one, two, four and eight warps a row, whole 16 bytes and ragged, and rows that no count of teams divides
@pytest.mark.parametrize("rows,d", [(9001, 136), (7001, 387), (5003, 1283), (4999, 1288), (3001, 2560), (3001, 2561), (2003, 5120),
                                    (2003, 5123), (1301, 10239), (1301, 10240)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_parameter_gradients_over_many_rows(wb, rows, d, kind, residual):
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    x, dy, dt = (torch.randn(rows, d, generator=g, device=DEV).to(TYPES[kind]) for _ in range(3))
    gamma = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    _, total, stats = wb.layernorm_forward(x, gamma, torch.zeros_like(gamma))
    _, dg, db = wb.layernorm_backward(dy, total, gamma, stats, dtotal=dt if residual else None)
    assert wb.check_device_error() == 0
    _check(dg, db, x, stats, dy, rows)


def test_parameter_gradients_past_32_bits(wb):
    # only rows around and behind the offset of 2^31 elements have a gradient: zeros add exactly
    rows, d, far = (1 << 31) // 1280 + 1000, 1280, 3000
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 1 << 18):
        x[i:i + (1 << 18)].normal_()
    dy = torch.zeros_like(x)
    dy[-far:].normal_()
    gamma = torch.rand(d, device=DEV)
    _, total, stats = wb.layernorm_forward(x, gamma, torch.zeros_like(gamma))
    _, dg, db = wb.layernorm_backward(dy, total, gamma, stats)
    assert wb.check_device_error() == 0
    _check(dg, db, x[-far:], stats[-far:], dy[-far:], far)


@pytest.mark.parametrize("d", [2559, 2561, 3519, 3521, 5119, 5121, 5631, 5633])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_ragged_forward_where_its_form_changes(wb, d, kind, residual):
    rows, t = 700, TYPES[kind]
    x, res, g, b, dy, _ = _inputs(rows, d, t, d, residual)
    y, total, stats = wb.layernorm_forward(x, g, b, 1e-5, residual=res)
    assert wb.check_device_error() == 0
    if residual:
        assert torch.equal(total, (x.float() + res.float()).to(t))
    want, mu, rs, _, _, _, _ = _reference(total, g, b, 1e-5, dy, None)
    # bounds of the forward pass as in test_gpu_layernorm_train
    xa = total.double().abs()
    ma = xa.mean(1, keepdim=True)
    _close(stats[:, 0], mu, 2.0 ** -23, 2.0 ** -19 * ma[:, 0])
    _close(stats[:, 1], rs, 2.0 ** -18, 2.0 ** -18 * ma[:, 0] * rs * rs)
    _close(y, want, torch.finfo(t).eps / 2,
           2.0 ** -18 * (g.double().abs() * rs[:, None] * (xa + ma) * (1 + ma * rs[:, None]) + b.double().abs()))
