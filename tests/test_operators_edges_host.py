"""CPU checks of the operators around the NVFP4 linear: what their entry points
refuse beyond single arguments, and host code that a GPU test cannot make fail."""
import ctypes

import pytest

P, i64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    return pkg.load()


def test_split_timeout_hook_takes_a_cta_or_off(lib):
    f = lib.gnq_inject_split_timeout
    assert f(8) == 2 and f(-2) == 2
    assert f(7) == 0 and f(-1) == 0
