"""Host-side refusals of the 4-bit entry points: an error code before any launch (no GPU needed)."""

import ctypes

import pytest

from compressed_sparse_kv_compress_b200 import _lib, build

nul = None


def _p(v=0x1000):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_mxfp4_validation(lib):
    def quant(x=_p(), dt=1, rows=4, D=64, codes=_p(), scale=_p(0x1001)):
        return lib.mxfp4_quantize(x, dt, rows, D, codes, scale, nul)

    def deq(codes=_p(), scale=_p(0x1001), rows=4, D=64, dt=1, out=_p()):
        return lib.mxfp4_dequantize(codes, scale, rows, D, dt, out, nul)

    for f in (quant, deq):
        assert f(rows=-1) == _lib.ERR_INVALID_ARG
        assert f(D=0) == _lib.ERR_INVALID_ARG
        assert f(D=48) == _lib.ERR_INVALID_ARG                  # half a block
        assert f(D=-32) == _lib.ERR_INVALID_ARG
        assert f(rows=1 << 40, D=32) == _lib.ERR_INVALID_ARG    # beyond the grid
        assert f(rows=(1 << 62), D=1 << 44) == _lib.ERR_INVALID_ARG
        assert f(dt=2) == _lib.ERR_UNSUPPORTED
        assert f(dt=7) == _lib.ERR_INVALID_ARG
        assert f(codes=nul) == _lib.ERR_INVALID_ARG
        assert f(scale=nul) == _lib.ERR_INVALID_ARG
        assert f(codes=_p(0x1008)) == _lib.ERR_INVALID_ARG
        assert f(rows=0, codes=nul) == _lib.OK
    assert quant(x=_p(0x1004)) == _lib.ERR_INVALID_ARG
    assert deq(out=nul) == _lib.ERR_INVALID_ARG


def test_kv4_validation(lib):
    def quant(rows=_p(), dt=0, n=4, lst=nul, cap=4, cache=_p()):
        return lib.kv_quantize_fp4(rows, dt, n, lst, cap, cache, nul, nul)

    def deq(rows=_p(), dt=0, n=4, lst=nul, cap=4, cache=_p()):
        return lib.kv_dequantize_fp4(cache, lst, cap, n, dt, rows, nul, nul)

    for f in (quant, deq):
        assert f(n=-1) == _lib.ERR_INVALID_ARG
        assert f(n=(1 << 35) + 1, cap=1 << 40) == _lib.ERR_INVALID_ARG
        assert f(cap=-1, lst=_p()) == _lib.ERR_INVALID_ARG
        assert f(cap=3) == _lib.ERR_INVALID_ARG                 # fewer cache rows than rows, no list
        assert f(dt=2) == _lib.ERR_UNSUPPORTED
        assert f(dt=-1) == _lib.ERR_INVALID_ARG
        assert f(rows=nul) == _lib.ERR_INVALID_ARG
        assert f(cache=nul) == _lib.ERR_INVALID_ARG
        assert f(cache=_p(0x1008)) == _lib.ERR_INVALID_ARG
        assert f(rows=_p(0x1008)) == _lib.ERR_INVALID_ARG
        assert f(lst=_p(0x1004)) == _lib.ERR_INVALID_ARG        # list not 8-byte aligned
        assert f(n=0, rows=nul, cache=nul) == _lib.OK


def test_matmul_validation(lib):
    def mm(a=_p(), ae=_p(0x1001), b=_p(), be=_p(0x1003), M=4, N=4, K=64, dt=1, out=_p()):
        return lib.mxfp4_matmul(a, ae, b, be, M, N, K, dt, out, nul, nul)

    assert mm(M=-1) == _lib.ERR_INVALID_ARG
    assert mm(N=-1) == _lib.ERR_INVALID_ARG
    assert mm(K=0) == _lib.ERR_INVALID_ARG
    assert mm(K=48) == _lib.ERR_INVALID_ARG
    assert mm(M=(1 << 30) + 1) == _lib.ERR_INVALID_ARG
    assert mm(K=(1 << 30) + 32) == _lib.ERR_INVALID_ARG
    assert mm(dt=2) == _lib.ERR_UNSUPPORTED
    assert mm(dt=5) == _lib.ERR_INVALID_ARG
    for name in ("a", "ae", "b", "be", "out"):
        assert mm(**{name: nul}) == _lib.ERR_INVALID_ARG
    for name in ("a", "b", "out"):
        assert mm(**{name: _p(0x1008)}) == _lib.ERR_INVALID_ARG
    assert mm(M=0, a=nul) == _lib.OK and mm(N=0, b=nul) == _lib.OK


def test_attention_flags(lib):
    def call(mode, T=0, out=_p(), noalloc=False, dtype=1):
        args = [mode, _p(), _p(), _p(), _p(), 8, _p(), _p(), nul, 128, nul, 0.1, _p(), _p(), 1, T, 16, 128, dtype, 100,
                out, nul]
        if noalloc:
            return lib.hybrid_decode_attn_noalloc(*args, nul, nul)
        return lib.hybrid_decode_attn(*args, _p(), 1 << 20, nul, nul)

    for na in (False, True):
        for m in (0, 1):
            assert call(m | _lib.ATTN_KV_FP4, noalloc=na) == _lib.OK
            assert call(m | _lib.ATTN_OUT_BF16 | _lib.ATTN_KV_FP8, noalloc=na) == _lib.OK
            assert call(m | _lib.ATTN_KV_FP4 | _lib.ATTN_OUT_BF16 | _lib.ATTN_PAIRS, noalloc=na) == _lib.OK
            assert call(m | _lib.ATTN_KV_FP4 | _lib.ATTN_KV_FP8, noalloc=na) == _lib.ERR_INVALID_ARG
            # outputs that are stored in wide words
            assert call(m | _lib.ATTN_KV_FP4, T=1, out=_p(0x1004), noalloc=na) == _lib.ERR_INVALID_ARG
            assert call(m | _lib.ATTN_OUT_BF16, T=1, out=_p(0x1008), noalloc=na) == _lib.ERR_INVALID_ARG
        assert call(7 | _lib.ATTN_KV_FP4, noalloc=na) == _lib.ERR_INVALID_ARG
