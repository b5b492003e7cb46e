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
    need = lib.wb_layernorm_backward_workspace_bytes(4, 64)
    assert need >= 2 * 64 * 4
    assert bwd(n=need - 1) == L.WB_EWORKSPACE
    assert lib.wb_layernorm_backward_workspace_bytes(0, 64) == 0
    assert lib.wb_layernorm_backward_workspace_bytes(4, 20000) == 0
    # the partial rows of the parameter gradients stop growing with the rows
    assert lib.wb_layernorm_backward_workspace_bytes(1 << 20, 1280) == lib.wb_layernorm_backward_workspace_bytes(1 << 21, 1280)
