"""Host-side refusals of the 4-bit calls at their exact limits (no GPU needed: an error code or an exception
before any launch)."""

import ctypes

import pytest
import torch

from compressed_sparse_kv_compress_b200 import _lib, api, build


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


class _Calls:
    """Stands in for the library and the current device (CPU tensors are on device -1): counts calls."""

    def __init__(self, monkeypatch):
        self.made = 0
        monkeypatch.setattr(_lib, "_lib", self)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)

    def hybrid_decode_attn(self, *args):
        self.made += 1
        return _lib.OK


class _Stream:
    cuda_stream = 0


def _attn_args():
    T, B, H, k = 3, 2, 4, 8
    return dict(q=torch.zeros(T, H, 128, dtype=torch.bfloat16), kv_cmp=torch.zeros(10, 176, dtype=torch.uint8),
                cmp_off=torch.zeros(B + 1, dtype=torch.int64), kv_raw=torch.zeros(7, 256, dtype=torch.bfloat16),
                raw_off=torch.zeros(B + 1, dtype=torch.int64), q_seq=torch.zeros(T, dtype=torch.int32),
                q_pos=torch.zeros(T, dtype=torch.int64), out=torch.zeros(T, H, 128, dtype=torch.bfloat16),
                workspace=torch.zeros(64, dtype=torch.uint8), idx=torch.zeros(T, k, dtype=torch.int32),
                raw_tok0=torch.zeros(B, dtype=torch.int64), sink=torch.zeros(H), lse=torch.zeros(T, H),
                dev_status=torch.zeros(1, dtype=torch.int32))


def _attend(**changed):
    a = dict(_attn_args(), **changed)
    lead = [a.pop(x) for x in ("q", "kv_cmp", "cmp_off", "kv_raw", "raw_off", "q_seq", "q_pos", "out", "workspace")]
    return api.hybrid_decode_attn(api.CSA, *lead, window=4, kv_fp4=True, stream=_Stream, **a)


def test_attention_arrays_that_the_kernels_would_misread(monkeypatch):
    """Every array's type, count and device: a narrower or shorter one would be read past its end."""
    calls = _Calls(monkeypatch)
    _attend()
    _attend(raw_tok0=None, sink=None, lse=None, dev_status=None, workspace=None)
    _attend(out=torch.zeros(3, 4, 128))
    assert calls.made == 3
    wrong = dict(
        q=[torch.zeros(3, 4, 128, dtype=torch.float16)], kv_cmp=[torch.zeros(10, 256, dtype=torch.bfloat16)],
        kv_raw=[torch.zeros(7, 256), torch.zeros(7, 128, dtype=torch.bfloat16)],
        out=[torch.zeros(3, 4, 64), torch.zeros(3, 4, 128, dtype=torch.float16)],
        cmp_off=[torch.zeros(3, dtype=torch.int32)], raw_off=[torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)],
        q_seq=[torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)],
        q_pos=[torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)],
        idx=[torch.zeros(3, 8, dtype=torch.int64), torch.zeros(2, 8, dtype=torch.int32)],
        raw_tok0=[torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)],
        sink=[torch.zeros(4, dtype=torch.bfloat16), torch.zeros(3)], lse=[torch.zeros(3, 4, dtype=torch.float64), torch.zeros(2, 4)],
        dev_status=[torch.zeros(1)])
    for name, values in wrong.items():
        for v in values:
            with pytest.raises(ValueError, match=name):
                _attend(**{name: v})
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)   # every tensor is elsewhere then
    with pytest.raises(ValueError, match="current device"):
        _attend()
    assert calls.made == 3


def test_attention_arrays_with_holes(monkeypatch):
    calls = _Calls(monkeypatch)
    for name, t in _attn_args().items():
        if name in ("workspace", "dev_status"):
            continue
        wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
        with pytest.raises(ValueError, match="contiguous"):
            _attend(**{name: wide})
    assert calls.made == 0
