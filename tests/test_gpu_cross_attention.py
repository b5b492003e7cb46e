"""Cross attention, forward and backward (GPU), against float64 evaluations of its formulas.

How far a result may be off is computed beside it.  A product of 64 terms is a sum in fp32: off by 2^-18 of
its terms' magnitude.  exp(s - max) then is off by the error of the two scores, 2^-21 of their size (the difference, its
scale and the exponential round in fp32) and 2^-20; it is rounded to bf16 (half a step, 2^-8) as a factor of p v and of dv,
and so is the gradient of the scores for dq and dk.  Every sum over keys or rows is off by 2^-18 of its
terms' magnitude again, and the results are rounded to bf16 (2^-8)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = 1.01 * 2.0 ** -8
SUM = 2.0 ** -18


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _data(batch, Tq, Tk, H, Hk, seed, sharp=1.0):
    g = _gen(seed)
    q = (torch.randn(batch, Tq, 64 * H, generator=g, device=DEV) * sharp).to(torch.bfloat16)
    kv = torch.randn(batch, Tk, 128 * Hk, generator=g, device=DEV).to(torch.bfloat16)
    dout = torch.randn(batch, Tq, 64 * H, generator=g, device=DEV).to(torch.bfloat16)
    return q, kv[..., :64 * Hk], kv[..., 64 * Hk:], dout, g


def _reference(q, k, v, dout, scale=0.125, q_lens=None, kv_lens=None):
    """name -> (value, how far it may be off), in the layout of the results."""
    batch, Tq, Tk = q.shape[0], q.shape[1], k.shape[1]
    H, Hk = q.shape[2] // 64, k.shape[2] // 64
    G = H // Hk
    f64 = dict(dtype=torch.float64, device=DEV)
    z = {n: (torch.zeros(s, **f64), torch.zeros(s, **f64)) for n, s in (
        ("out", (batch, Tq, H, 64)), ("dq", (batch, Tq, H, 64)), ("dk", (batch, Tk, Hk, 64)), ("dv", (batch, Tk, Hk, 64)))}
    z["lse"] = (torch.full((batch, H, Tq), -math.inf, **f64), torch.zeros(batch, H, Tq, **f64))
    for i in range(batch):
        a = Tq if q_lens is None else min(max(int(q_lens[i]), 0), Tq)
        b = Tk if kv_lens is None else min(max(int(kv_lens[i]), 0), Tk)
        if a == 0 or b == 0:
            continue
        qi = q[i, :a].double().view(a, Hk, G, 64).permute(1, 2, 0, 3)          # [Hk, G, a, 64]
        ki = k[i, :b].double().reshape(b, Hk, 1, 64).permute(1, 2, 0, 3)
        vi = v[i, :b].double().reshape(b, Hk, 1, 64).permute(1, 2, 0, 3)
        s = scale * (qi @ ki.mT)
        es = SUM * scale * (qi.abs() @ ki.abs().mT)
        lse = torch.logsumexp(s, -1, keepdim=True)
        es_row = es.amax(-1, keepdim=True)
        size = s.abs().amax(-1, keepdim=True) + lse.abs() + 1
        rel = torch.expm1(2 * es_row + 2.0 ** -21 * size + 2.0 ** -20)
        p = torch.exp(s - lse)
        out = p @ vi
        e_out = (HALF + 2 * rel + SUM) * (p @ vi.abs()) + HALF * out.abs()
        e_lse = es_row + 2.0 ** -20 * size
        put = lambda n, value, off, rows: (z[n][0][i, :rows].copy_(value), z[n][1][i, :rows].copy_(off))  # noqa: E731
        heads = lambda x: x.permute(2, 0, 1, 3).reshape(a, H, 64)  # noqa: E731
        put("out", heads(out), heads(e_out), a)
        z["lse"][0][i, :, :a] = lse.reshape(H, a)
        z["lse"][1][i, :, :a] = e_lse.reshape(H, a)
        if dout is None:
            continue
        do = dout[i, :a].double().view(a, Hk, G, 64).permute(1, 2, 0, 3)
        dp = do @ vi.mT
        e_dp = SUM * (do.abs() @ vi.abs().mT)
        delta = (do * out).sum(-1, keepdim=True)
        e_delta = (do.abs() * (e_out + SUM * out.abs())).sum(-1, keepdim=True)
        rel = rel + torch.expm1(e_lse)                                        # the lse that it takes is the forward pass's
        ds = p * (dp - delta)
        e_ds = (HALF + rel) * ds.abs() + (1 + rel) * p * (e_dp + e_delta + 2.0 ** -22 * (dp.abs() + delta.abs()))
        dq = scale * (ds @ ki)
        put("dq", heads(dq), heads(scale * ((e_ds + SUM * ds.abs()) @ ki.abs()) + HALF * dq.abs() + 1e-30), a)
        keys = lambda x: x.sum(1).permute(1, 0, 2)  # noqa: E731
        dk = keys(scale * (ds.mT @ qi))
        put("dk", dk, keys(scale * ((e_ds + SUM * ds.abs()).mT @ qi.abs())) + HALF * dk.abs() + 1e-30, b)
        dv = keys(p.mT @ do)
        put("dv", dv, keys(((HALF + rel + SUM) * p).mT @ do.abs()) + HALF * dv.abs() + 1e-30, b)
    return {n: (x, e) if n == "lse" else (x.flatten(2), e.flatten(2)) for n, (x, e) in z.items()}


def _check(got, ref):
    for name, t in got.items():
        value, off = ref[name]
        g = t.double()
        assert g.shape == value.shape, name
        none = value == -math.inf
        assert bool((g[none] == -math.inf).all()), name
        g, value, off = g[~none], value[~none], off[~none]
        assert bool(torch.isfinite(g).all()), name
        if g.numel():
            over = (g - value).abs() - off
            assert float(over.max()) <= 0, (name, float(over.max()), float(((g - value).abs() / off.clamp(min=1e-300)).max()))


def _both(wb, q, k, v, dout, **kw):
    out, lse = wb.cross_attention(q, k, v, **kw)
    dq, dk, dv = wb.cross_attention_backward(dout, q, k, v, out, lse, **kw)
    assert wb.check_device_error() == 0
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# rows of a key head of 1 to 16 and more take different kernels, and sides of up to 64 rows or keys others in the backward pass; tiles are
# 128 rows and keys
SHAPES = [(1, 1, 1, 1, 1), (2, 1, 1500, 3, 3), (1, 5, 16, 2, 2), (3, 4, 17, 4, 1), (2, 16, 129, 2, 2), (1, 17, 40, 2, 2), (2, 8, 300, 8, 2),
          (1, 32, 1000, 1, 1), (1, 33, 127, 1, 1), (2, 64, 128, 2, 2), (1, 65, 64, 3, 3), (1, 127, 65, 2, 1), (2, 128, 129, 2, 2),
          (1, 129, 1, 2, 2), (2, 200, 257, 6, 2), (1, 448, 1500, 2, 2), (3, 77, 1371, 2, 2), (1, 300, 63, 4, 4), (40, 1, 50, 4, 4)]


@pytest.mark.parametrize("batch,Tq,Tk,H,Hk", SHAPES)
@pytest.mark.parametrize("sharp", [0.3, 4.0])
def test_against_float64(wb, batch, Tq, Tk, H, Hk, sharp):
    q, k, v, dout, _ = _data(batch, Tq, Tk, H, Hk, Tq + Tk, sharp)
    _check(_both(wb, q, k, v, dout), _reference(q, k, v, dout))


@pytest.mark.parametrize("batch,Tq,Tk,H,Hk", [(5, 1, 333, 2, 2), (5, 3, 40, 8, 4), (5, 20, 200, 2, 2), (5, 130, 300, 2, 1), (5, 70, 129, 2, 2)])
def test_lengths_and_what_lies_behind_them(wb, batch, Tq, Tk, H, Hk):
    # NaN and infinities behind the lengths reach nothing; no rows, no keys, one of each, lengths outside 0..T
    q, k, v, dout, g = _data(batch, Tq, Tk, H, Hk, Tk)
    q_lens = torch.tensor([Tq, 0, max(1, Tq // 2), Tq + 7, 1], dtype=torch.int32, device=DEV)
    kv_lens = torch.tensor([Tk // 2, Tk, 0, 1, Tk + 9], dtype=torch.int32, device=DEV)
    ref = _reference(q, k, v, dout, q_lens=q_lens, kv_lens=kv_lens)
    for bad in (math.nan, math.inf, -math.inf, 3e38):
        q2, k2, v2, d2 = (t.clone() for t in (q, k, v, dout))
        for i in range(batch):
            a, b = min(int(q_lens[i]), Tq), min(int(kv_lens[i]), Tk)
            q2[i, a:], d2[i, a:], k2[i, b:], v2[i, b:] = bad, bad, bad, bad
        _check(_both(wb, q2, k2, v2, d2, q_lens=q_lens, kv_lens=kv_lens), ref)


@pytest.mark.parametrize("Tq", [3, 150])
@pytest.mark.parametrize("end", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193])
def test_lengths_inside_tiles(wb, Tq, end):
    q, k, v, dout, _ = _data(2, Tq, 200, 2, 2, end)
    k[:, end:] = math.nan
    v[:, end:] = math.nan
    lens = torch.full((2,), end, dtype=torch.int32, device=DEV)
    rows = torch.tensor([min(end, Tq), Tq], dtype=torch.int32, device=DEV)
    _check(_both(wb, q, k, v, dout, q_lens=rows, kv_lens=lens), _reference(q, k, v, dout, q_lens=rows, kv_lens=lens))


@pytest.mark.parametrize("Tq", [2, 130])
def test_strides(wb, Tq):
    # rows cut from wider ones, items apart, one state for the whole batch; a dimension of one with any stride
    H, Hk, Tk, batch = 4, 2, 150, 3
    q, k, v, dout, g = _data(batch, Tq, Tk, H, Hk, 7)
    want = _both(wb, q, k.contiguous(), v.contiguous(), dout)
    _check(want, _reference(q, k, v, dout))
    wide = torch.randn(batch, Tq + 3, 3 * 64 * H + 8, device=DEV).to(torch.bfloat16)
    wide[:, 1:Tq + 1, 8:8 + 64 * H] = q
    wide[:, 1:Tq + 1, 8 + 64 * H:8 + 128 * H] = dout
    got = _both(wb, wide[:, 1:Tq + 1, 8:8 + 64 * H], k, v, wide[:, 1:Tq + 1, 8 + 64 * H:8 + 128 * H])
    seq = torch.empty(Tq, batch, 64 * H, dtype=torch.bfloat16, device=DEV)
    seq.copy_(q.transpose(0, 1))
    got2 = _both(wb, seq.transpose(0, 1), k, v, dout)
    for name in want:
        assert torch.equal(want[name], got[name]) and torch.equal(want[name], got2[name]), name
    one_k, one_v = k[:1].expand(batch, -1, -1), v[:1].expand(batch, -1, -1)
    got = _both(wb, q, one_k, one_v, dout)
    want = _both(wb, q, one_k.contiguous(), one_v.contiguous(), dout)
    for name in want:
        assert torch.equal(want[name], got[name]), name
    one = _both(wb, q[:1].as_strided((1, Tq, 64 * H), (5, 64 * H, 1)), k[:1], v[:1], dout[:1])
    want = _both(wb, q[:1].clone(), k[:1].contiguous(), v[:1].contiguous(), dout[:1])
    for name in want:
        assert torch.equal(want[name], one[name]), name


@pytest.mark.parametrize("Tq", [4, 140])
@pytest.mark.parametrize("size", [2.0 ** 12, 1e15])
def test_large_scores(wb, Tq, size):
    # scores on a grid, exact in fp32, far apart: the softmax is one key's, or even among the same largest ones
    g = _gen(3)
    q = torch.zeros(1, Tq, 64, device=DEV)
    k = torch.zeros(1, 200, 64, device=DEV)
    q[..., 0] = size
    k[..., 0] = torch.randint(-4, 5, (1, 200), generator=g, device=DEV).float()
    v, dout = torch.randn(1, 200, 64, generator=g, device=DEV), torch.randn(1, Tq, 64, generator=g, device=DEV)
    q, k, v, dout = (t.to(torch.bfloat16) for t in (q, k, v, dout))
    got = _both(wb, q, k, v, dout)
    first = (k[0, :, 0] == k[0, :, 0].max())
    mean = v[0, first].double().mean(0)
    n = int(first.sum())
    top = float(q[0, 0, 0]) * float(k[0, :, 0].max()) / 8
    # each p is 1 in bf16 and exact; sums of n terms and the quotient round, then the result
    assert bool(((got["out"].double() - mean).abs() <= HALF * mean.abs() + SUM * v[0, first].double().abs().mean(0)).all())
    assert bool(((got["lse"].double() - (top + math.log(n))).abs() <= 2.0 ** -22 * top + 2.0 ** -20).all())
    assert bool(torch.isfinite(got["dq"]).all()) and bool(torch.isfinite(got["dk"]).all())
    assert not got["dv"][0, ~first].any() and not got["dk"][0, ~first].any()
    if size < 1e6:                                                # lse holds log n to 2^-11 there, and p is off by as much
        dv = dout[0].double().sum(0) / n
        off = (HALF + 2.0 ** -10) * (dout[0].double().abs().sum(0) / n) + HALF * dv.abs()
        assert bool(((got["dv"][0, first].double() - dv).abs() <= off).all())


@pytest.mark.parametrize("Tq", [4, 140])
def test_scores_of_minus_infinity(wb, Tq):
    # a row with some scores of -infinity is the softmax of the others, wherever they lie; one with nothing else has no softmax
    q, k, v, dout, _ = _data(1, Tq, 300, 1, 1, 5)
    q[..., 0] = 1
    k[..., 0] = 0
    k[0, :200, 0] = -math.inf
    out, lse = wb.cross_attention(q, k, v)
    ref = _reference(q, k[:, 200:], v[:, 200:], None)
    _check({"out": out, "lse": lse}, ref)
    k[..., 0] = -math.inf
    out, lse = wb.cross_attention(q, k, v)
    assert wb.check_device_error() == 0
    assert bool(torch.isnan(out).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("batch,Tq,Tk,H,Hk", [(4, 1, 1500, 8, 8), (3, 9, 700, 8, 2), (2, 64, 900, 4, 4), (2, 33, 500, 4, 1)])
def test_gradients_of_few_rows_are_rounded_once(wb, batch, Tq, Tk, H, Hk):
    # Half a step is 2^-8 of a value at most, so one rounding that spreads evenly is off by no more than 2^-8 / sqrt(3) of the values' norm
    # (near 1.6 of 2.26 thousandths, since most values lie above a power of two).  P and dS rounded to bf16 too would add as much again
    # in squares: 2.3 to 2.6 thousandths.
    q, k, v, dout, _ = _data(batch, Tq, Tk, H, Hk, 31 + Tq)
    got, ref = _both(wb, q, k, v, dout), _reference(q, k, v, dout)
    for name in ("dk", "dv"):
        off = float((got[name].double() - ref[name][0]).norm() / ref[name][0].norm())
        assert off < 2.0 ** -8 / math.sqrt(3), (name, off)


@pytest.mark.parametrize("Tq,Tk", [(150, 300), (40, 2500), (200, 60)])
def test_keys_with_a_large_common_part(wb, Tq, Tk):
    # dq = scale sum_k dS k, and sum_k dS = 0: what all keys share takes no part.  The kernel subtracts (sum_k dS) M, M = sum_k P k, from what it
    # sums, dS rounded in both, so whatever dS is off by adds up along k - M: half a step, P's relative error and the errors of dP and
    # delta.  Along k itself: the sums in fp32, and M's P being rounded, times the sum of dS.
    q, k, v, dout, _ = _data(2, Tq, Tk, 2, 2, 7 + Tk)
    k = k.clone()
    k.view(2, Tk, 2, 64)[..., :8] += 48
    got = _both(wb, q, k, v, dout)
    heads = lambda x: x.double().view(2, -1, 2, 64).transpose(1, 2)  # noqa: E731
    qh, kh, vh, do = heads(q), heads(k), heads(v), heads(dout)
    s = 0.125 * (qh @ kh.mT)
    es = 2 * SUM * 0.125 * (qh.abs() @ kh.abs().mT).amax(-1, keepdim=True)
    p = torch.softmax(s, -1)
    rel = torch.expm1(2 * es + 2.0 ** -20 * (2 * s.abs().amax(-1, keepdim=True) + 10))
    out = p @ vh
    e_delta = (do.abs() * (2 * HALF + 3 * rel) * (p @ vh.abs())).sum(-1, keepdim=True)
    ds = p * (do @ vh.mT - (do * out).sum(-1, keepdim=True))
    e_ds = (HALF + rel) * ds.abs() + (1 + rel) * p * (SUM * (do.abs() @ vh.abs().mT) + e_delta)
    m = p @ kh
    dq = 0.125 * (ds @ kh)
    sum_ds = e_ds.sum(-1, keepdim=True)
    away = torch.cat([(e_ds[:, :, t:t + 50, :, None] * (kh[:, :, None] - m[:, :, t:t + 50, None]).abs()).sum(-2) for t in range(0, Tq, 50)], 2)
    off = 0.125 * (away + SUM * (ds.abs() @ kh.abs()) + sum_ds * (HALF + 2 * SUM) * (p @ kh.abs())) + HALF * dq.abs()
    over = (heads(got["dq"]) - dq).abs() / off
    assert float(over.max()) <= 1, float(over.max())


@pytest.mark.parametrize("Tq,Tk", [(1, 1), (5, 1), (150, 1), (70, 64), (150, 1500)])
def test_one_key(wb, Tq, Tk):
    # its weight is 1 whatever q and k are: no gradient reaches them, and out is its v
    q, k, v, dout, _ = _data(3, Tq, Tk, 4, 2, Tq, 4.0)
    lens = torch.tensor([1, Tk, 1], dtype=torch.int32, device=DEV)
    got = _both(wb, q, k, v, dout, kv_lens=lens)
    _check(got, _reference(q, k, v, dout, kv_lens=lens))
    for i in (0, 2):
        assert not got["dq"][i].any() and not got["dk"][i].any()
        assert torch.equal(got["out"][i].view(Tq, 2, 2, 64), v[i, :1].reshape(1, 2, 1, 64).expand(Tq, 2, 2, 64))


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -20, 0.07])
@pytest.mark.parametrize("Tq", [6, 100])
def test_scales(wb, scale, Tq):
    q, k, v, dout, _ = _data(2, Tq, 180, 2, 2, 9)
    _check(_both(wb, q, k, v, dout, scale=scale), _reference(q, k, v, dout, scale=scale))


def test_nothing_to_do(wb):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    out, lse = wb.cross_attention(z(0, 4, 128), z(0, 5, 64), z(0, 5, 64))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 2, 4)
    for Tq in (3, 50):
        got = _both(wb, z(2, Tq, 128), z(2, 0, 64), z(2, 0, 64), z(2, Tq, 128))
        assert not got["out"].any() and bool((got["lse"] == -math.inf).all()) and not got["dq"].any() and got["dk"].shape == (2, 0, 64)
    got = _both(wb, z(2, 0, 128), z(2, 7, 64), z(2, 7, 64), z(2, 0, 128))
    assert got["out"].shape == (2, 0, 128) and not got["dk"].any() and not got["dv"].any()


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
def test_gradients_that_are_not_needed(wb, need):
    q, k, v, dout, _ = _data(2, 90, 200, 2, 1, 3)
    out, lse = wb.cross_attention(q, k, v)
    whole = wb.cross_attention_backward(dout, q, k, v, out, lse)
    part = wb.cross_attention_backward(dout, q, k, v, out, lse, need_dq=need[0], need_dkv=need[1])
    for a, b, n in zip(whole, part, (need[0], need[1], need[1])):
        assert (b is None) == (not n) and (b is None or torch.equal(a, b))


def test_gradients_against_differences(wb):
    # the directional derivative of sum(dout out) in 64 bits, central differences of the formula, against the kernel's gradients
    q, k, v, dout, g = _data(1, 40, 70, 2, 2, 21)
    got = _both(wb, q, k, v, dout)

    def f(q, k, v):
        h = lambda t: t.view(1, -1, 2, 64).transpose(1, 2)  # noqa: E731
        p = torch.softmax(h(q) @ h(k).mT / 8, -1)
        return ((p @ h(v)).transpose(1, 2).reshape(dout.shape) * dout.double()).sum()

    args = [t.double().contiguous() for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        step = torch.randn(args[i].shape, dtype=torch.float64, generator=g, device=DEV)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * step, args[i] - 1e-5 * step
        want = float(f(*up) - f(*down)) / 2e-5
        # the error bounds of the elements, along the step, and 1e-6 for the differences' third order
        off = float((_reference(q, k, v, dout)[name][1] * step.abs()).sum())
        assert abs(float((got[name].double() * step).sum()) - want) <= off + 1e-6 * float(step.abs().sum())


@pytest.mark.parametrize("batch,Tq,Tk,H,Hk", [(1, 1, 1500, 20, 20), (2, 7, 700, 8, 2), (2, 200, 500, 4, 2)])
def test_same_call_same_bits_and_captured(wb, batch, Tq, Tk, H, Hk):
    q, k, v, dout, _ = _data(batch, Tq, Tk, H, Hk, 11)
    first = _both(wb, q, k, v, dout)
    torch.empty(1 << 28, dtype=torch.uint8, device=DEV).fill_(0xFF)
    again = _both(wb, q, k, v, dout)
    side = torch.cuda.Stream()
    on_side = {}
    out, lse = wb.cross_attention(q, k, v, stream=side)
    on_side["dq"], on_side["dk"], on_side["dv"] = wb.cross_attention_backward(dout, q, k, v, out, lse, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = wb.cross_attention(q, k, v)
        dq, dk, dv = wb.cross_attention_backward(dout, q, k, v, out, lse)
    for _ in range(3):
        for t in (out, lse, dq, dk, dv):
            t.fill_(7)
        graph.replay()
    for name, t in dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv).items():
        assert torch.equal(first[name], again[name]) and torch.equal(first[name], t), name
        assert name not in on_side or torch.equal(first[name], on_side[name]), name
    assert wb.check_device_error() == 0


def test_results_do_not_depend_on_the_rest_of_a_batch_of_many_rows(wb):
    # too few keys for the rule that splits them where a batch has few tiles
    q, k, v, dout, _ = _data(3, 150, 300, 2, 2, 13)
    whole = _both(wb, q, k, v, dout)
    part = _both(wb, q[1:2], k[1:2], v[1:2], dout[1:2])
    for name in whole:
        assert torch.equal(whole[name][1:2], part[name]), name


def test_offsets_past_32_bits(wb):
    # more than 2^31 elements of K and V: the last item against the same item alone
    batch, Tk, d = 800, 1500, 1280
    kv = torch.empty(batch, Tk, 2 * d, dtype=torch.bfloat16, device=DEV)
    for i in range(0, batch, 100):
        kv[i:i + 100].normal_()
    k, v = kv[..., :d], kv[..., d:]
    for Tq in (1, 40):
        q = torch.randn(batch, Tq, d, device=DEV).to(torch.bfloat16)
        dout = torch.randn(batch, Tq, d, device=DEV).to(torch.bfloat16)
        got = _both(wb, q, k, v, dout)
        ref = _reference(q[-1:], k[-1:], v[-1:], dout[-1:])
        _check({n: t[-1:] for n, t in got.items()}, ref)
        del got


def test_python_refusals(wb):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    q, k = z(2, 3, 128), z(2, 5, 64)
    out, lse = wb.cross_attention(q, k, k)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: wb.cross_attention(q.float(), k, k), lambda: wb.cross_attention(q[0], k, k), lambda: wb.cross_attention(z(2, 3, 96), k, k),
                lambda: wb.cross_attention(q, z(1, 5, 64), z(1, 5, 64)), lambda: wb.cross_attention(q, z(2, 5, 192), z(2, 5, 192)),
                lambda: wb.cross_attention(q, k, z(2, 6, 64)), lambda: wb.cross_attention(q.transpose(1, 2).contiguous().transpose(1, 2), k, k),
                lambda: wb.cross_attention(q, k, k, q_lens=lens.long()), lambda: wb.cross_attention(q, k, k, kv_lens=lens[:1]),
                lambda: wb.cross_attention(q, k, k, kv_lens=lens.cpu()), lambda: wb.cross_attention(q, z(2, 5, 64).cpu(), k),
                lambda: wb.cross_attention_backward(q[:1], q, k, k, out, lse), lambda: wb.cross_attention_backward(q, q, k, k, out[:, :2], lse),
                lambda: wb.cross_attention_backward(q, q, k, k, out, lse[:, :1])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: wb.cross_attention(q, k, k, scale=0.0), lambda: wb.cross_attention(q, k, k[:1].expand(2, -1, -1)),
                lambda: wb.cross_attention(z(2, 3, 132)[..., 2:130], k, k),
                lambda: wb.cross_attention_backward(q, q, k, k, out, lse, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(wb.WbError):
            bad()
    assert wb.check_device_error() == 0


# few tiles of rows: clusters of 4 and 8 CTAs split the keys, 8 the ones of few rows
@pytest.mark.parametrize("batch,Tq,Tk,H,Hk", [(5, 130, 1500, 2, 1), (5, 40, 3000, 2, 2), (5, 3, 1500, 2, 2), (5, 256, 2000, 1, 1)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 3e38])
def test_what_lies_behind_the_lengths_of_split_keys(wb, batch, Tq, Tk, H, Hk, bad):
    # keys that end inside a CTA's last tile, at its border, and in the first tile, so that the other CTAs of a cluster have none
    q, k, v, dout, g = _data(batch, Tq, Tk, H, Hk, Tk + Tq)
    q_lens = torch.tensor([Tq, Tq - 1, max(1, Tq // 2), 1, Tq + 3], dtype=torch.int32, device=DEV)
    for ends in ([Tk // 2 + 3, 100, 1, Tk - 1, 129], [Tk, 128, 0, 127, 640], [383, 257, Tk + 9, 1023, 511]):
        kv_lens = torch.tensor(ends, dtype=torch.int32, device=DEV)
        ref = _reference(q, k, v, dout, q_lens=q_lens, kv_lens=kv_lens)
        q2, k2, v2, d2 = (t.clone() for t in (q, k, v, dout))
        for i in range(batch):
            a, b = min(int(q_lens[i]), Tq), min(int(kv_lens[i]), Tk)
            q2[i, a:], d2[i, a:], k2[i, b:], v2[i, b:] = bad, bad, bad, bad
        got = _both(wb, q2, k2, v2, d2, q_lens=q_lens, kv_lens=kv_lens)
        _check(got, ref)
        kw = dict(q_lens=q_lens, kv_lens=kv_lens)
        dq, none, _ = wb.cross_attention_backward(d2, q2, k2, v2, got["out"], got["lse"], need_dkv=False, **kw)
        none2, dk, dv = wb.cross_attention_backward(d2, q2, k2, v2, got["out"], got["lse"], need_dq=False, **kw)
        assert none is None and none2 is None
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            assert torch.equal(t, got[name]), name
    assert wb.check_device_error() == 0
