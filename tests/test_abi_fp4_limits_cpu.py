"""Host-side refusals of the 4-bit calls at their exact limits (no GPU needed: an error code or an exception
before any launch)."""

import ctypes

import pytest

from compressed_sparse_kv_compress_b200 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_values_beyond_the_grid(lib):
    """A CTA takes 8192 values and a grid 2^31 - 1 CTAs: 2^44 - 8192 values at most."""
    p = ctypes.c_void_p(0x1000)
    most = ((1 << 31) - 1) * 8192
    for rows, D in ((1 << 39, 32), (1, 1 << 44), (most // 32 + 1, 32), (1, most + 32), ((most + 64) // 64, 64)):
        assert rows * D > most and rows * D <= 1 << 44
        assert lib.mxfp4_quantize(p, 1, rows, D, p, p, None) == _lib.ERR_INVALID_ARG
        assert lib.mxfp4_dequantize(p, p, rows, D, 1, p, None) == _lib.ERR_INVALID_ARG
