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


def test_scratch_of_a_decode_is_what_the_header_says(L):
    """With weights about 4 B H capacity bytes, heads in even parts of at most
    16 a kv head; without, no more than 8.6 MB whatever the shape."""
    size = L.thrift_kv8_decode_workspace_size
    for B, H, Hkv, cap in ((64, 64, 8, 131072), (4, 32, 8, 8192), (3, 7, 1, 40000), (2, 38, 2, 5000)):
        G = H // Hkv
        parts = -(-G // 16)
        even = -(-G // parts) + 1 & ~1
        for d in (64, 128):
            scores = 4 * B * Hkv * parts * even * cap
            assert 0 < size(B, H, Hkv, cap, d, 0) <= 8_600_000
            more = size(B, H, Hkv, cap, d, 1) - size(B, H, Hkv, cap, d, 0)
            assert scores <= more <= scores + 8 * B * H + 512
