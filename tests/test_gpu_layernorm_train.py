"""LayerNorm for training (GPU): forward with row statistics and backward with the parameter gradients,
against float64 evaluations of the formulas.

Tolerances count roundings: an output rounded once to its type is off by half a step, eps / 2 relative
to itself; what is summed in fp32 is off by a few 2^-24 of the magnitudes that enter the sum, counted
as 2^-19 (32 of them) for a row's terms and as sqrt(rows) + 16 of them for the sums over rows."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _inputs(rows, d, t, seed, residual):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x = (2 * n(rows, d) + 0.3).to(t)
    res = n(rows, d).to(t) if residual else None
    return x, res, 1 + 0.1 * n(d), 0.1 * n(d), n(rows, d).to(t), (n(rows, d).to(t) if residual else None)


def _reference(total, g, b, eps, dy, dt):
    x, g, b, dy = total.double(), g.double(), b.double(), dy.double()
    mu = x.mean(1, keepdim=True)
    rs = 1 / ((x - mu) ** 2).mean(1, keepdim=True).add(eps).sqrt()
    h = (x - mu) * rs
    u = dy * g
    dx = rs * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    if dt is not None:
        dx = dx + dt.double()
    # magnitudes that the fp32 sums and differences go through
    mag = rs * (u.abs() + u.abs().mean(1, keepdim=True) + h.abs() * (u * h).abs().mean(1, keepdim=True))
    mag = mag + rs * (x.abs() + x.abs().mean(1, keepdim=True)) * rs * (u * h).abs().mean(1, keepdim=True)
    return h * g + b, mu[:, 0], rs[:, 0], dx, (dy * h).sum(0), dy.sum(0), mag


def _close(got, ref, half_step, absolute):
    got = got.double()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    ok = err <= half_step * ref.abs() * (1 + 2.0 ** -6) + absolute
    assert bool(ok.all()), float((err - half_step * ref.abs() - absolute).max())


SHAPES = [(1, 1), (3, 7), (5, 8), (1, 1280), (2, 256), (7, 264), (129, 384), (33, 1283), (600, 640), (65, 1288),
          (17, 2560), (9, 2564), (1500, 1280), (50, 5120), (21, 5127), (3, 10240), (4, 9001)]


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_and_backward_match_the_formulas(wb, rows, d, kind, residual):
    t = TYPES[kind]
    half = torch.finfo(t).eps / 2
    x, res, g, b, dy, dt = _inputs(rows, d, t, rows * 31 + d, residual)
    y, total, stats = wb.layernorm_forward(x, g, b, 1e-5, residual=res)
    assert wb.check_device_error() == 0
    if residual:
        assert torch.equal(total, (x.float() + res.float()).to(t))
    else:
        assert total is x
    dx, dg, db = wb.layernorm_backward(dy, total, g, stats, dtotal=dt)
    assert wb.check_device_error() == 0
    ry, mu, rs, rdx, rdg, rdb, mag = _reference(total, g, b, 1e-5, dy, dt)
    xa = total.double().abs()
    # mean: 2^-19 of the row's mean magnitude; rstd: twice that against the spread, plus 2 ulp of rsqrt
    _close(stats[:, 0], mu, 2.0 ** -23, 2.0 ** -19 * xa.mean(1))
    _close(stats[:, 1], rs, 2.0 ** -18, 2.0 ** -18 * xa.mean(1) * rs * rs)
    slack = 2.0 ** -18 * (g.double().abs() * rs[:, None] * (xa + xa.mean(1, keepdim=True)) * (1 + xa.mean(1, keepdim=True) * rs[:, None])
                          + b.double().abs()) + (6e-8 if kind == "f16" else 0)
    _close(y, ry, half, slack)
    tiny = 6e-8 if kind == "f16" else 0.0           # f16 values below 2^-14 step by 2^-24
    grow = (1 + xa.mean(1, keepdim=True) * rs[:, None])
    _close(dx, rdx, half, 2.0 ** -18 * (mag * grow + (dt.double().abs() if residual else 0)) + tiny)
    n_sum = 2.0 ** -24 * (rows ** 0.5 + 16) * 4
    hmag = (total.double().abs() + mu[:, None].abs()) * rs[:, None]
    _close(dg, rdg, 0.0, (n_sum + 2.0 ** -20) * (dy.double().abs() * hmag * grow).sum(0) + 1e-30)
    _close(db, rdb, 0.0, n_sum * dy.double().abs().sum(0) + 1e-30)


# more rows than the device holds at once: every slot is filled several times over
@pytest.mark.parametrize("rows,d", [(20011, 136), (15001, 1280), (12007, 1928), (7001, 4104), (4003, 10240),
                                    (3001, 1283), (20011, 387), (9001, 1021), (6001, 5123), (2503, 10239)])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
def test_a_row_does_not_depend_on_the_rows_around_it(wb, rows, d, kind, residual):
    x, res, g, b, dy, dt = _inputs(rows, d, TYPES[kind], d, residual)
    y, total, stats = wb.layernorm_forward(x, g, b, residual=res)
    dx, _, _ = wb.layernorm_backward(dy, total, g, stats, dtotal=dt, need_params=False)
    assert wb.check_device_error() == 0
    cut = lambda t, a: None if t is None else t[a:a + 100].clone()  # noqa: E731
    for at in (0, 1187, rows // 2, rows - 100):
        ys, ts, ss = wb.layernorm_forward(cut(x, at), g, b, residual=cut(res, at))
        ds, _, _ = wb.layernorm_backward(cut(dy, at), ts, g, ss, dtotal=cut(dt, at), need_params=False)
        for whole, part in ((y, ys), (total, ts), (stats, ss), (dx, ds)):
            assert torch.equal(whole[at:at + 100], part)


def test_backward_matches_differences_of_the_forward(wb):
    # directional derivative of sum(dy . y) + sum(dt . total) along random directions, f32
    rows, d = 6, 96
    x, res, g, b, dy, dt = _inputs(rows, d, torch.float32, 5, True)
    _, total, stats = wb.layernorm_forward(x, g, b, 1e-5, residual=res)
    dx, dg, db = wb.layernorm_backward(dy, total, g, stats, dtotal=dt)
    gen = torch.Generator(device=DEV).manual_seed(9)
    vx, vg, vb = (torch.randn(s, generator=gen, device=DEV) for s in ((rows, d), (d,), (d,)))

    def value(e):
        y, tot, _ = wb.layernorm_forward(x + e * vx, g + e * vg, b + e * vb, 1e-5, residual=res)
        return float((dy.double() * y.double()).sum() + (dt.double() * tot.double()).sum())

    h = 2.0 ** -7
    slope = (value(h) - value(-h)) / (2 * h)
    want = float((dx.double() * vx).sum() + (dg.double() * vg).sum() + (db.double() * vb).sum())
    # each value sums 2 * rows * d terms of size ~1 rounded at 2^-22, over 2 h; third derivatives times h^2 / 6
    scale = float((dx.double() * vx).abs().sum() + (dg.double() * vg).abs().sum() + (db.double() * vb).abs().sum())
    assert abs(slope - want) < 2.0 ** -22 * (2 * rows * d) ** 0.5 * 8 / (2 * h) + h * h * scale


def test_parameter_gradients_are_the_same_every_time_and_may_be_left_out(wb):
    x, _, g, b, dy, _ = _inputs(4099, 1280, torch.bfloat16, 3, False)
    _, total, stats = wb.layernorm_forward(x, g, b)
    first = wb.layernorm_backward(dy, total, g, stats)
    again = wb.layernorm_backward(dy, total, g, stats)
    for a, c in zip(first, again):
        assert torch.equal(a, c)
    dx, dg, db = wb.layernorm_backward(dy, total, g, stats, need_params=False)
    assert dg is None and db is None and torch.equal(dx, first[0])


def test_no_rows(wb):
    x = torch.empty(0, 384, device=DEV)
    g, b = torch.ones(384, device=DEV), torch.zeros(384, device=DEV)
    y, total, stats = wb.layernorm_forward(x, g, b)
    assert y.shape == (0, 384) and stats.shape == (0, 2)
    dx, dg, db = wb.layernorm_backward(x, x, g, stats)
    assert dx.shape == (0, 384) and not dg.any() and not db.any()


@pytest.mark.parametrize("d", [1280, 1283, 5120])
def test_dx_may_overwrite_an_input(wb, d):
    from whisper_encoder_gb300 import _lib
    x, _, g, b, dy, dt = _inputs(3001, d, torch.bfloat16, 8, True)
    _, total, stats = wb.layernorm_forward(x, g, b)
    want, _, _ = wb.layernorm_backward(dy, total, g, stats, dtotal=dt, need_params=False)
    for which in range(3):
        a = [dy.clone(), total.clone(), dt.clone()]
        p = [t.data_ptr() for t in a]
        _lib.call("wb_layernorm_backward", p[0], p[1], g.data_ptr(), stats.data_ptr(), p[2], 3001, d, _lib.WB_BF16,
                  p[which], None, None, None, 0, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(a[which], want)


def test_not_a_number_stays_in_its_row(wb):
    x, _, g, b, dy, _ = _inputs(40, 512, torch.bfloat16, 11, False)
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    y, total, stats = wb.layernorm_forward(x, g, b)
    dx, _, _ = wb.layernorm_backward(dy, total, g, stats)
    bad = torch.zeros(40, dtype=torch.bool, device=DEV)
    bad[[7, 9]] = True
    assert torch.equal(torch.isnan(y).all(1), bad) and torch.equal(torch.isnan(y).any(1), bad)
    assert torch.equal(torch.isnan(dx).all(1), bad) and torch.equal(torch.isnan(dx).any(1), bad)


def test_on_a_side_stream_and_in_a_graph(wb):
    x, res, g, b, dy, dt = _inputs(777, 640, torch.bfloat16, 2, True)

    def both(stream=None):
        y, total, stats = wb.layernorm_forward(x, g, b, residual=res, stream=stream)
        return (y, *wb.layernorm_backward(dy, total, g, stats, dtotal=dt, stream=stream))

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, c in zip(want, got):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(both(), got):
        assert torch.equal(a, c)


def test_refusals(wb):
    x, res, g, b, dy, _ = _inputs(4, 64, torch.bfloat16, 1, True)
    y, total, stats = wb.layernorm_forward(x, g, b)
    for bad in (lambda: wb.layernorm_forward(x.double(), g, b),
                lambda: wb.layernorm_forward(x[:, ::2], g[:32].contiguous(), b[:32].contiguous()),
                lambda: wb.layernorm_forward(x, g[:32], b),
                lambda: wb.layernorm_forward(x, g.half(), b),
                lambda: wb.layernorm_forward(x, g, b, residual=res.float()),
                lambda: wb.layernorm_forward(x, g, b, residual=res[:2]),
                lambda: wb.layernorm_forward(x.cpu(), g, b),
                lambda: wb.layernorm_backward(dy[:2], total, g, stats),
                lambda: wb.layernorm_backward(dy, total, g, stats[:2]),
                lambda: wb.layernorm_backward(dy.float(), total, g, stats)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(wb.WbError):
        wb.layernorm_forward(x, g, b, eps=0.0)
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(wb.WbError):                                   # base not on 16 bytes
        wb.layernorm_forward(flat[1:].view(4, 64), g, b)
    wide = torch.zeros(1, 10241, device=DEV)
    with pytest.raises(wb.WbError):
        wb.layernorm_forward(wide, wide[0].clone(), wide[0].clone())
