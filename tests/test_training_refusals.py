"""CPU checks of the training entry points: sizes, pointers and workspaces are refused on the host,
before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from whisper_encoder_gb300 import build
    build.build()
    from whisper_encoder_gb300 import _lib
    return _lib.load()


OTHER = ctypes.c_void_p(1 << 21)
FAKE = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 2)


def test_layernorm_train_refusals(lib):
    from whisper_encoder_gb300 import _lib as L

    def fwd(x=FAKE, res=None, g=FAKE, b=FAKE, rows=4, d=64, eps=1e-5, dtype=L.WB_BF16, y=FAKE, total=None, stats=FAKE):
        return lib.wb_layernorm_forward(x, res, g, b, rows, d, eps, dtype, y, total, stats, None)

    def bwd(dy=FAKE, x=FAKE, g=FAKE, stats=FAKE, dt=None, rows=4, d=64, dtype=L.WB_F32, dx=FAKE, dg=FAKE, db=FAKE,
            ws=FAKE, n=1 << 30):
        return lib.wb_layernorm_backward(dy, x, g, stats, dt, rows, d, dtype, dx, dg, db, ws, n, None)

    assert fwd(rows=0, x=None) == L.WB_OK
    assert bwd(rows=0, dy=None, dg=None, db=None) == L.WB_OK
    for f in (fwd, bwd):
        assert f(dtype=L.WB_E4M3) == L.WB_EUNSUPPORTED
        assert f(dtype=9) == L.WB_EUNSUPPORTED
        assert f(rows=-1) == L.WB_EINVAL
        assert f(d=0) == L.WB_EINVAL
        assert f(d=10241) == L.WB_EINVAL
        for name in ("x", "g", "stats"):
            assert f(**{name: None}) == L.WB_EINVAL
            assert f(**{name: ODD}) == L.WB_EINVAL
    assert fwd(eps=0.0) == L.WB_EINVAL
    assert fwd(eps=float("nan")) == L.WB_EINVAL
    assert fwd(res=FAKE) == L.WB_EINVAL                 # a residual without a place for the sum
    assert fwd(total=FAKE) == L.WB_EINVAL
    assert bwd(dx=None) == L.WB_EINVAL
    assert bwd(dt=ODD) == L.WB_EINVAL
    assert bwd(dg=None) == L.WB_EINVAL                  # one parameter gradient without the other
    assert bwd(ws=None) == L.WB_EWORKSPACE
    need = lib.wb_layernorm_backward_workspace_bytes(4, 64, L.WB_F32)
    assert need >= 2 * 64 * 4
    assert bwd(n=need - 1) == L.WB_EWORKSPACE
    assert lib.wb_layernorm_backward_workspace_bytes(0, 64, L.WB_F32) == 0
    assert lib.wb_layernorm_backward_workspace_bytes(4, 20000, L.WB_F32) == 0
    assert lib.wb_layernorm_backward_workspace_bytes(4, 64, L.WB_E4M3) == 0
    # the partial rows of the parameter gradients stop growing with the rows
    assert (lib.wb_layernorm_backward_workspace_bytes(1 << 20, 1280, L.WB_BF16)
            == lib.wb_layernorm_backward_workspace_bytes(1 << 21, 1280, L.WB_BF16))


def test_head_loss_refusals(lib):
    from whisper_encoder_gb300 import _lib as L
    BIG = 1 << 40

    def ce(x=FAKE, w=FAKE, labels=FAKE, M=8, d=64, V=100, e=0.0, loss=FAKE, lse=FAKE, ws=FAKE, n=BIG):
        return lib.wb_linear_cross_entropy(x, w, labels, M, d, V, e, loss, lse, ws, n, None)

    def ce_bwd(dloss=FAKE, x=FAKE, w=FAKE, labels=FAKE, lse=FAKE, M=8, d=64, V=100, e=0.0, dx=OTHER, dw=OTHER, ws=FAKE, n=BIG):
        return lib.wb_linear_cross_entropy_backward(dloss, x, w, labels, lse, M, d, V, e, dx, dw, ws, n, None)

    def kl(x=FAKE, w=FAKE, top=FAKE, ty=L.WB_F32, index=FAKE, M=8, d=64, V=100, k=4, T=1.0, loss=FAKE, lse=FAKE, ws=FAKE, n=BIG):
        return lib.wb_linear_distill(x, w, top, ty, index, M, d, V, k, T, loss, lse, ws, n, None)

    def kl_bwd(dloss=FAKE, x=FAKE, w=FAKE, top=FAKE, ty=L.WB_F32, index=FAKE, lse=FAKE, M=8, d=64, V=100, k=4, T=1.0, dx=OTHER,
               dw=OTHER, ws=FAKE, n=BIG):
        return lib.wb_linear_distill_backward(dloss, x, w, top, ty, index, lse, M, d, V, k, T, dx, dw, ws, n, None)

    for f in (ce, ce_bwd, kl, kl_bwd):
        for name, value in (("M", -1), ("M", (1 << 24) + 1), ("d", 0), ("d", 12), ("d", 65544), ("V", 0), ("V", (1 << 24) + 1),
                            ("x", None), ("x", ODD), ("w", None), ("w", ODD), ("lse", None), ("lse", ODD)):
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
        assert f(ws=None) == L.WB_EWORKSPACE
        assert f(ws=ODD) == L.WB_EWORKSPACE
    for f in (ce, ce_bwd):
        for name, value in (("labels", None), ("labels", ODD), ("e", -0.5), ("e", 1.0), ("e", float("nan"))):
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
    for f in (kl, kl_bwd):
        for name, value in (("top", None), ("top", ODD), ("index", None), ("index", ODD), ("k", 0), ("k", 1025), ("T", 0.0), ("T", -1.0),
                            ("T", float("nan")), ("T", float("inf"))):
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
        assert f(ty=L.WB_E4M3) == L.WB_EUNSUPPORTED
    for f in (ce_bwd, kl_bwd):
        for name, value in (("dloss", None), ("dloss", ODD), ("dx", ODD), ("dw", ODD)):
            assert f(**{name: value}) == L.WB_EINVAL, (f, name, value)
        assert f(dx=None, dw=None, x=OTHER, w=OTHER) == L.WB_OK       # nothing wanted, nothing launched
        assert f(dx=OTHER, x=OTHER) == L.WB_EINVAL and f(dw=OTHER, w=OTHER) == L.WB_EINVAL   # a gradient over its input
    assert ce(M=0, x=None, labels=None, ws=None) == L.WB_OK
    assert kl(M=0, x=None, top=None, ws=None) == L.WB_OK
    assert ce_bwd(M=0, x=None, labels=None, ws=None, dw=None) == L.WB_OK
    assert kl_bwd(M=0, x=None, top=None, ws=None, dw=None) == L.WB_OK
    # one byte less than the query says
    for f, q, shape in ((ce, lib.wb_linear_cross_entropy_workspace_bytes, (8, 64, 100)),
                        (ce_bwd, lib.wb_linear_cross_entropy_backward_workspace_bytes, (8, 64, 100)),
                        (kl, lib.wb_linear_distill_workspace_bytes, (8, 64, 100, 4)),
                        (kl_bwd, lib.wb_linear_distill_backward_workspace_bytes, (8, 64, 100, 4))):
        assert f(n=q(*shape) - 1) == L.WB_EWORKSPACE
        assert q(0, *shape[1:]) == 0 and q(-1, *shape[1:]) == 0 and q(8, 60, *shape[2:]) == 0


def test_head_workspace_does_not_grow_with_the_logits(lib):
    # twice the vocabulary at many rows: the backward pass keeps a piece, not M x V
    small = lib.wb_linear_cross_entropy_backward_workspace_bytes(16384, 1280, 50000)
    large = lib.wb_linear_cross_entropy_backward_workspace_bytes(16384, 1280, 100000)
    assert large == small and small < 16384 * 50000 * 2
    # the forward pass keeps statistics per 256 columns
    assert lib.wb_linear_cross_entropy_workspace_bytes(16384, 1280, 50000) < 16384 * (50000 // 16 + 1280 * 2 + 64)
