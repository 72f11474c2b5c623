"""Pins of oracle/kv4.py: 4-bit main-KV rows built byte by byte, exact round trips, ties,
saturation, zero and non-finite blocks, and the element formats' error bounds."""

import numpy as np
import pytest

from oracle import codecs, kv4


def test_hand_built_row_decodes_to_known_values():
    row = np.zeros((1, kv4.ROW_BYTES), dtype=np.uint8)
    row[0, kv4.OFF_SCALE:kv4.OFF_SCALE + 8] = [127, 128, 127, 126, 130, 127, 127, 127]
    row[0, 0] = 0x92            # dims 0, 1: codes 2 and 9 -> 1.0, -0.5
    row[0, 16] = 0x07           # dim 32: code 7 -> 6 x 2
    row[0, 32] = 0x38           # dim 64: E4M3 1.0
    row[0, 64] = 0xBC           # dim 96: E4M3 -1.5, scale 1/2
    row[0, 96] = 0xF0           # dim 129 (V dim 1): code 15 -> -6 x 8
    v = kv4.decode_rows(row)[0]
    want = {0: 1.0, 1: -0.5, 32: 12.0, 64: 1.0, 96: -0.75, 129: -48.0}
    for i in range(256):
        assert v[i] == want.get(i, 0.0), i


def test_representable_rows_round_trip():
    rng = np.random.default_rng(3)
    v = rng.choice([0, .5, 1, 1.5, 2, 3, 4, 6], (64, 8, 32)) * rng.choice([-1, 1], (64, 8, 32))
    v[:, :, 0] = 6.0                                  # pins the shared exponent of E2M1 blocks
    v[:, 2:4] = np.where(np.arange(32) == 0, 448.0, np.round(v[:, 2:4]) * 16)
    v *= np.ldexp(1.0, rng.integers(-100, 100, (64, 8)))[..., None]
    rows = v.reshape(64, 256)
    assert np.array_equal(kv4.decode_rows(kv4.quantize_rows_f64(rows)), rows)


def test_zero_ties_saturation_and_non_finite_blocks():
    rows = np.zeros((5, 256))
    p = kv4.quantize_rows_f64(rows)
    assert not p.any()                                # a zero row is all zero bytes
    rows[1, :6] = [4.0, 0.25, 0.75, 2.5, 5.0, -7.5]   # scale 1: 0.25 -> 0, 0.75 -> 1, 2.5 -> 2, 5 -> 4, -7.5 -> -6
    rows[2, 64:67] = [448.0, 500.0, -511.0]           # E4M3 at scale 1: both saturate
    rows[3, 130] = np.inf
    rows[3, 200] = 1.0
    rows[4, 70] = np.nan
    d = kv4.decode_rows(kv4.quantize_rows_f64(rows))
    assert np.array_equal(d[1, :6], [4.0, 0.0, 1.0, 2.0, 4.0, -6.0])
    assert np.array_equal(d[2, 64:67], [448.0, 448.0, -448.0])
    assert np.isnan(d[3, 128:160]).all() and d[3, 200] == 1.0 and np.isfinite(d[3, :128]).all()
    assert np.isnan(d[4, 64:96]).all() and np.isfinite(d[4, 96:]).all()


@pytest.mark.parametrize("seed", [0, 1])
def test_error_bounds(seed):
    """E2M1: half a step of 2 (a quarter of 4..6), or the saturation from below 8 to 6, against a
    scale with amax in [4, 8): |error| <= 2 scale <= amax / 2.  E4M3: half a step is 2^-4 relative,
    or the saturation from below 512 to 448 (1/8), or half a subnormal step of the scale."""
    rng = np.random.default_rng(seed)
    rows = rng.standard_normal((256, 256)) * np.exp(rng.uniform(-20, 20, (256, 1)))
    d = np.abs(kv4.decode_rows(kv4.quantize_rows_f64(rows)) - rows).reshape(256, 8, 32)
    b = np.abs(rows).reshape(256, 8, 32)
    amax = b.max(-1, keepdims=True)
    for i in range(8):
        if i in kv4.ROPE_BLOCKS:
            assert np.all(d[:, i] <= np.maximum(b[:, i] / 8, amax[:, i] * 2.0 ** -18))
        else:
            assert np.all(d[:, i] <= amax[:, i] / 2)


def test_rows_match_the_vector_codec():
    """Blocks of E2M1 elements are those of the MXFP4 vectors."""
    rng = np.random.default_rng(7)
    rows = rng.standard_normal((32, 256))
    c, s = codecs.mx_fp4_quantize(rows[:, 128:])
    p = kv4.quantize_rows_f64(rows)
    assert np.array_equal(p[:, kv4.OFF_V:kv4.OFF_SCALE], codecs.pack_nibbles(c))
    assert np.array_equal(p[:, kv4.OFF_SCALE + 4:kv4.OFF_SCALE + 8], s)
