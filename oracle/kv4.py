"""4-bit main-KV rows: the compressed cache in OCP microscaling formats, the position-sensitive
dimensions at a higher precision (test infrastructure: only tests/ and the smoke check use it).

[SW] shareware.cn/news/167317 §十三.4 (and §六.1): low-bit storage is enough for ranking and for
most dimensions, while the dimensions more sensitive to position keep a higher precision; it gives
no format.  The reading taken here follows the FP8 rows (oracle/kv8.py) and the MXFP4 indexer
vectors (oracle/codecs.py):

* A compressed row is K (128 dims) then V (128 dims): eight blocks of 32 values, each with one E8M0
  scale 2^(e - 127).
* K's last 64 dimensions (blocks 2 and 3), the position-encoded ones, are E4M3 elements (MXFP8:
  shared exponent floor(log2 amax) - 8); the other six blocks are E2M1 (MXFP4: minus 2).  The
  shared exponent is at least -127; a block of zeros takes the smallest scale.
* A block that holds an infinity or a NaN takes e = 255 (NaN) and zero codes.
* Storage, 176 bytes a row: K dims 0..63 (32 B, element 2j in the low nibble) | K dims 64..127
  (64 B) | V (64 B) | the eight scale codes | 8 zero bytes."""

from __future__ import annotations

import numpy as np

from . import codecs

ROW_BYTES = 176
OFF_K, OFF_ROPE, OFF_V, OFF_SCALE = 0, 32, 96, 160
E4M3_EMAX = 8
ROPE_BLOCKS = (2, 3)


def shared_exponent(x: np.ndarray, emax: int) -> np.ndarray:
    """floor(log2(amax)) - emax of each row of x [..., 32], clamped to [-127, 127]."""
    amax = np.max(np.abs(np.asarray(x, dtype=np.float64)), axis=-1)
    _, e2 = np.frexp(np.where(amax > 0, amax, 1.0))
    return np.clip(np.where(amax > 0, e2 - 1 - emax, -127), -127, 127)


def quantize_rows_f64(rows: np.ndarray) -> np.ndarray:
    """K||V rows [N, 256] -> storage rows [N, 176] uint8, every step exact in float64 before the
    one rounding of each element."""
    r = np.asarray(rows, dtype=np.float64).reshape(-1, 8, 32)
    bad = ~np.isfinite(r).all(axis=-1)
    r = np.where(bad[..., None], 0.0, r)
    n = r.shape[0]
    out = np.zeros((n, ROW_BYTES), dtype=np.uint8)
    codes = np.zeros((n, 8, 32), dtype=np.uint8)
    for b in range(8):
        rope = b in ROPE_BLOCKS
        e = shared_exponent(r[:, b], E4M3_EMAX if rope else codecs.E2M1_EMAX)
        y = r[:, b] / np.ldexp(1.0, e)[:, None]
        codes[:, b] = codecs.e4m3_encode(y) if rope else codecs.e2m1_encode(y)
        out[:, OFF_SCALE + b] = (e + 127).astype(np.uint8)
    codes[bad] = 0
    out[:, OFF_SCALE:OFF_SCALE + 8][bad] = 0xFF
    out[:, OFF_K:OFF_ROPE] = codecs.pack_nibbles(codes[:, :2].reshape(n, 64))
    out[:, OFF_ROPE:OFF_V] = codes[:, 2:4].reshape(n, 64)
    out[:, OFF_V:OFF_SCALE] = codecs.pack_nibbles(codes[:, 4:].reshape(n, 128))
    return out


def decode_rows(packed: np.ndarray) -> np.ndarray:
    """Storage rows [N, 176] -> K||V values [N, 256] float64 (exact)."""
    p = np.asarray(packed, dtype=np.uint8)
    n = p.shape[0]
    v = np.concatenate([codecs.e2m1_decode(codecs.unpack_nibbles(p[:, OFF_K:OFF_ROPE])),
                        codecs.e4m3_decode(p[:, OFF_ROPE:OFF_V]),
                        codecs.e2m1_decode(codecs.unpack_nibbles(p[:, OFF_V:OFF_SCALE]))], axis=1)
    s = codecs.e8m0_decode(p[:, OFF_SCALE:OFF_SCALE + 8])
    return (v.reshape(n, 8, 32) * s[..., None]).reshape(n, 256)
