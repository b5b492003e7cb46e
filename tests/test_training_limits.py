"""CPU checks of the limits of the training entry points: temperatures, workspaces."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(1 << 20)            # aligned, never dereferenced on these paths
OTHER = ctypes.c_void_p(1 << 21)


@pytest.fixture(scope="module")
def lib():
    from whisper_encoder_gb300 import build
    build.build()
    from whisper_encoder_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("T", [1e-40, 2.0 ** -127, float("inf"), float("nan")])
def test_temperatures_without_a_finite_reciprocal_are_refused(lib, T):
    from whisper_encoder_gb300 import _lib as L
    n = 1 << 40
    assert lib.wb_linear_distill(FAKE, FAKE, FAKE, L.WB_F32, FAKE, 8, 64, 100, 4, T, FAKE, FAKE, FAKE, n, None) == L.WB_EINVAL
    assert lib.wb_linear_distill_backward(FAKE, FAKE, FAKE, FAKE, L.WB_F32, FAKE, FAKE, 8, 64, 100, 4, T, OTHER, OTHER, FAKE, n,
                                          None) == L.WB_EINVAL
    # without rows too
    assert lib.wb_linear_distill(None, FAKE, None, L.WB_F32, None, 0, 64, 100, 4, T, None, None, None, 0, None) == L.WB_EINVAL


@pytest.mark.parametrize("M,d,V", [(1, 64, 1 << 24), (17, 64, 1 << 24), (129, 1280, 1_000_000), (257, 384, 1_000_000), (4480, 1280, 1 << 20)])
def test_a_piece_of_the_gradient_stays_within_its_bound(lib, M, d, V):
    # the piece of softmax - target takes 2^28 bytes at most, whole tiles of rows included; what else there is: x and
    # x' in 16 bits, float32 slabs of dx (together at most 152 tiles of 128 x 256 or as many tiles as dx has), row maps
    rows = -(-M // 256) * 256
    slabs = max(152 * 128 * 256, rows * (d + 256)) * 4
    rest = 2 * rows * d * 2 + slabs + 64 * M + 4096
    assert lib.wb_linear_cross_entropy_backward_workspace_bytes(M, d, V) <= (1 << 28) + rest


def test_layernorm_pointers_are_aligned_as_the_header_says(lib):
    from whisper_encoder_gb300 import _lib as L
    at = lambda n: ctypes.c_void_p((1 << 20) + n)  # noqa: E731

    def fwd(x=FAKE, res=OTHER, g=FAKE, b=FAKE, y=FAKE, total=FAKE, stats=FAKE, d=7):
        return lib.wb_layernorm_forward(x, res, g, b, 4, d, 1e-5, L.WB_BF16, y, total, stats, None)

    def bwd(dy=FAKE, x=FAKE, g=FAKE, stats=FAKE, dt=FAKE, dx=FAKE, dg=FAKE, db=FAKE, ws=FAKE, d=7):
        return lib.wb_layernorm_backward(dy, x, g, stats, dt, 4, d, L.WB_BF16, dx, dg, db, ws, 1 << 30, None)

    for d in (7, 64):
        for name in ("x", "res", "g", "b", "y", "total"):
            assert fwd(**{name: at(8)}, d=d) == L.WB_EINVAL, name
        for name in ("dy", "x", "g", "dt", "dx", "dg", "db"):
            assert bwd(**{name: at(8)}, d=d) == L.WB_EINVAL, name
        assert bwd(ws=at(8), d=d) == L.WB_EWORKSPACE
        assert fwd(stats=at(4), d=d) == L.WB_EINVAL and bwd(stats=at(4), d=d) == L.WB_EINVAL
