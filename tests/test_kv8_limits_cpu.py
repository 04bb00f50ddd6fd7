"""The limits of the 8-bit cache's C ABI that the header states, without a
device: refused before any launch."""
import ctypes as C

import pytest

from bit_quantization_b200 import build, ops


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


P = C.c_void_p


def _decode(L, scale):
    return L.thrift_kv8_decode(P(1 << 20), 1, 2, 4, 2, 64, 16, 40, 5120, 2560, 64, P(1 << 21),
                               P(1 << 22), P(1 << 23), P(1 << 24), P(1 << 25), C.c_float(scale),
                               None, P(1 << 26), P(1 << 27), P(1 << 28), 1 << 40, None)


def test_a_scale_that_overflows_in_log2_units_is_refused(L):
    """scale log2 e is what multiplies the scores: from 2.36e38 on it is no
    fp32 number, and rows would be NaN."""
    for scale in (2.4e38, -2.4e38, 3.0e38, 3.4e38, float("inf"), float("nan")):
        assert _decode(L, scale) == ops.ERR_ARG, scale
