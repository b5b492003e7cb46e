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
