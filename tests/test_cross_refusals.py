"""CPU checks of cross attention, gradient clipping and the policy loss: sizes, strides, pointers, overlaps
and workspaces are refused on the host, before anything is launched."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from whisper_encoder_gb300 import build
    build.build()
    from whisper_encoder_gb300 import _lib
    return _lib.load()


def test_cross_attention_refusals(lib):
    from whisper_encoder_gb300 import _lib as L

    def fwd(q=FAKE, qb=512, qr=128, k=FAKE, kb=1024, kr=128, v=FAKE, vb=1024, vr=128, ql=None, kl=None, batch=2, Tq=4, Tk=8, H=2, Hk=1,
            scale=0.125, out=FAKE, lse=FAKE):
        return lib.wb_cross_attention(q, qb, qr, k, kb, kr, v, vb, vr, ql, kl, batch, Tq, Tk, H, Hk, scale, out, lse, None)

    def bwd(do=FAKE, db=512, dr=128, q=FAKE, qb=512, qr=128, k=FAKE, kb=1024, kr=128, v=FAKE, vb=1024, vr=128, out=FAKE, lse=FAKE,
            ql=None, kl=None, batch=2, Tq=4, Tk=8, H=2, Hk=1, scale=0.125, dq=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, n=BIG):
        return lib.wb_cross_attention_backward(do, db, dr, q, qb, qr, k, kb, kr, v, vb, vr, out, lse, ql, kl, batch, Tq, Tk, H, Hk, scale,
                                               dq, dk, dv, ws, n, None)

    for f in (fwd, bwd):
        assert f(batch=0, q=None, k=None, v=None) == L.WB_OK
        for name, value in (("batch", -1), ("Tq", -1), ("Tk", -1), ("Tq", (1 << 24) + 1), ("Tk", (1 << 24) + 1), ("H", 0), ("H", 3), ("Hk", 0),
                            ("Hk", 2), ("H", 2048), ("scale", 0.0), ("scale", -1.0), ("scale", float("nan")), ("scale", float("inf")),
                            ("scale", 2.0 ** -65), ("batch", 1 << 30),
                            ("q", None), ("q", ODD), ("k", None), ("k", ODD), ("v", None), ("v", ODD), ("out", None), ("out", ODD),
                            ("lse", None), ("lse", ODD), ("ql", ODD), ("kl", ODD),
                            ("qr", 120), ("qr", 132), ("qr", 1 << 38), ("kr", 56), ("kr", 68), ("vr", 0), ("qb", -512), ("qb", 516), ("kb", 4),
                            ("kb", 1 << 38), ("vb", 0)):      # one of k and v expanded over the batch
            if (name, value) == ("Hk", 2):
                assert f(Hk=2, kr=64) == L.WB_EINVAL          # rows shorter than the heads
                continue
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
    assert fwd(Tq=0, q=None) == L.WB_OK
    assert bwd(dq=None, dk=None, dv=None, q=None) == L.WB_OK          # nothing wanted
    for name, value in (("do", None), ("do", ODD), ("dr", 64), ("db", 4), ("dk", None), ("dv", None), ("dq", ODD), ("dk", ODD), ("dv", ODD)):
        assert bwd(**{name: value}) == L.WB_EINVAL, (name, value)
    need = lib.wb_cross_attention_backward_workspace_bytes(2, 4, 2)
    assert need == 2 * 2 * 128 * 8
    assert bwd(n=need - 1) == L.WB_EWORKSPACE and bwd(ws=None) == L.WB_EWORKSPACE and bwd(ws=ODD) == L.WB_EWORKSPACE
    assert lib.wb_cross_attention_backward_workspace_bytes(0, 4, 2) == 0
    assert lib.wb_cross_attention_backward_workspace_bytes(2, 0, 2) == 0


def test_clip_refusals(lib):
    from whisper_encoder_gb300 import _lib as L

    def clip(at=((1 << 20), (1 << 21)), outs=None, n=(64, 64), ty=(L.WB_F32, L.WB_BF16), oty=None, count=None, max_norm=1.0, norm=FAKE,
             ws=FAKE, nbytes=BIG, arrays=True):
        i64 = lambda x: None if x is None else (ctypes.c_int64 * len(x))(*x)  # noqa: E731
        i32 = lambda x: None if x is None else (ctypes.c_int32 * len(x))(*x)  # noqa: E731
        return lib.wb_clip_grad_norm(i64(at) if arrays else None, i64(outs), i64(n), i32(ty), i32(oty), len(at) if count is None else count,
                                     max_norm, norm, ws, nbytes, None)

    a, b = 1 << 20, 1 << 21
    ty = (L.WB_F32, L.WB_BF16)
    assert clip(count=-1) == L.WB_EINVAL and clip(count=L.WB_CLIP_MAX_TENSORS + 1) == L.WB_EINVAL
    assert clip(norm=None) == L.WB_EINVAL and clip(norm=ODD) == L.WB_EINVAL
    assert clip(arrays=False) == L.WB_EINVAL
    assert clip(ty=(L.WB_F32, L.WB_E4M3)) == L.WB_EUNSUPPORTED
    assert clip(n=(-1, 64)) == L.WB_EINVAL and clip(n=((1 << 40) + 1, 64)) == L.WB_EINVAL
    assert clip(at=(0, b)) == L.WB_EINVAL and clip(at=(a + 2, b)) == L.WB_EINVAL and clip(at=(a, b + 1)) == L.WB_EINVAL
    assert clip(ws=None) == L.WB_EWORKSPACE and clip(ws=ODD) == L.WB_EWORKSPACE
    need = lib.wb_clip_grad_norm_workspace_bytes(2)
    assert need > 0 and clip(nbytes=need - 1) == L.WB_EWORKSPACE
    assert lib.wb_clip_grad_norm_workspace_bytes(0) == 0
    assert lib.wb_clip_grad_norm_workspace_bytes(5000) > lib.wb_clip_grad_norm_workspace_bytes(500)
    # written tensors
    own = dict(outs=(a, b), oty=ty)
    for m in (-1.0, float("nan")):
        assert clip(max_norm=m, **own) == L.WB_EINVAL
    assert clip(outs=(a, b)) == L.WB_EINVAL                                        # no types
    assert clip(outs=(a, b), oty=(L.WB_BF16, L.WB_BF16)) == L.WB_EUNSUPPORTED        # narrower
    assert clip(outs=(a, b), oty=(L.WB_F32, L.WB_F16)) == L.WB_EUNSUPPORTED
    assert clip(outs=(a, b), oty=(L.WB_F32, L.WB_F32)) == L.WB_EINVAL               # in place into another type
    assert clip(outs=(a, 0), oty=ty) == L.WB_EINVAL and clip(outs=(a, 4 * b + 1), oty=ty) == L.WB_EINVAL
    assert clip(at=(a, a), n=(64, 64), ty=(L.WB_F32,) * 2, outs=(a, a), oty=(L.WB_F32,) * 2) == L.WB_EINVAL        # listed twice
    assert clip(at=(a, a + 252), n=(64, 64), ty=(L.WB_F32,) * 2, outs=(a, a + 252), oty=(L.WB_F32,) * 2) == L.WB_EINVAL
    assert clip(outs=(4 * b, 4 * b + 128), oty=ty) == L.WB_EINVAL                   # outputs over one another
    assert clip(outs=(b, 4 * b), oty=ty) == L.WB_EINVAL                             # an output over another gradient
    assert clip(outs=(a + 4, b), oty=ty) == L.WB_EINVAL                             # over its own, shifted
    assert clip(ws=None, **own) == L.WB_EWORKSPACE                                   # all else is right


def test_policy_refusals(lib):
    from whisper_encoder_gb300 import _lib as L

    def fwd(nll=FAKE, old=FAKE, ref=FAKE, adv=FAKE, tok=0, labels=FAKE, S=4, T=8, lo=0.2, hi=0.2, kl=0.1, seq=0, stats=FAKE, weight=FAKE,
            ws=FAKE, n=BIG):
        return lib.wb_policy_loss(nll, old, ref, adv, tok, labels, S, T, lo, hi, kl, seq, stats, weight, ws, n, None)

    def bwd(dloss=FAKE, nll=FAKE, old=FAKE, ref=FAKE, adv=FAKE, tok=0, labels=FAKE, weight=FAKE, S=4, T=8, lo=0.2, hi=0.2, kl=0.1,
            dnll=FAKE):
        return lib.wb_policy_loss_backward(dloss, nll, old, ref, adv, tok, labels, weight, S, T, lo, hi, kl, dnll, None)

    nan, inf = float("nan"), float("inf")
    for f in (fwd, bwd):
        for name, value in (("S", -1), ("T", -1), ("S", (1 << 31) + 1), ("T", (1 << 30) + 1), ("lo", -0.1), ("lo", 1.1), ("lo", nan), ("hi", -0.1),
                            ("hi", inf), ("hi", nan), ("kl", nan), ("kl", inf), ("nll", None), ("nll", ODD), ("old", None), ("old", ODD),
                            ("ref", ODD), ("ref", None), ("adv", None), ("adv", ODD), ("labels", None), ("labels", ODD), ("weight", None),
                            ("weight", ODD)):
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
        assert f(S=1 << 31, T=1 << 30) == L.WB_EINVAL
    assert fwd(stats=None) == L.WB_EINVAL and fwd(stats=ODD) == L.WB_EINVAL
    # one block's sizes need no workspace
    assert lib.wb_policy_loss_workspace_bytes(128, 512) == 0
    for S, T in ((129, 1), (1, 513), (4096, 448)):
        need = lib.wb_policy_loss_workspace_bytes(S, T)
        assert need > 0 and fwd(S=S, T=T, n=need - 1) == L.WB_EWORKSPACE
        assert fwd(S=S, T=T, ws=None) == L.WB_EWORKSPACE and fwd(S=S, T=T, ws=ODD) == L.WB_EWORKSPACE
    assert lib.wb_policy_loss_workspace_bytes(0, 8) == 0 and lib.wb_policy_loss_workspace_bytes(4, 0) == 0
    for name in ("dloss", "dnll"):
        assert bwd(**{name: None}) == L.WB_EINVAL and bwd(**{name: ODD}) == L.WB_EINVAL
    assert bwd(S=0, nll=None) == L.WB_OK and bwd(T=0, nll=None) == L.WB_OK


def test_python_entry_points_refuse_host_tensors():
    import whisper_encoder_gb300 as wb
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    x = torch.zeros(2, 3)
    for call in (lambda: wb.cross_attention(q, q, q), lambda: wb.grad_norm([x]), lambda: wb.grad_norm([]), lambda: wb.clip_grad_norm([x], 1.0),
                 lambda: wb.policy_loss(x, x, x[:, 0], x), lambda: wb.policy_loss(None, x, x[:, 0], x)):
        with pytest.raises(ValueError):
            call()


def test_order_of_dimensions_that_leaves_no_gaps():
    from whisper_encoder_gb300.api import _dense
    x = torch.zeros(4, 6, 5)
    assert _dense(x) and _dense(x.permute(2, 0, 1)) and _dense(x[:, :, :1].contiguous().transpose(0, 2)) and _dense(torch.zeros(0, 3).T)
    assert not _dense(x[:, :4]) and not _dense(x[::2]) and not _dense(torch.zeros(1, 5).expand(4, 5)) and not _dense(x[..., 0])
