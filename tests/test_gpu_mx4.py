"""MXFP4 vectors and 4-bit main-KV rows on the GPU: codes and scales equal those of the exact
definitions (oracle/codecs.py, oracle/kv4.py) byte for byte -- scales are powers of two, so both
sides round the same exact quotients -- and the inverses decode every byte exactly."""

import numpy as np
import pytest
import torch

from oracle import codecs, kv4

from compressed_sparse_kv_compress_b200 import CskvError, _lib, api
from helpers import to_f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _values(rng, n, D, dtype):
    """Rows over the whole range of magnitudes, with ties, zeros, subnormals and negative zeros."""
    x = rng.standard_normal((n, D)) * np.exp2(rng.integers(-40, 40, (n, 1)))
    x.reshape(-1)[::7] = 0.0
    x.reshape(-1)[3::11] *= 2.0 ** -6
    flat = x.reshape(-1, 32)
    flat[0] = 0.0
    if len(flat) > 6:
        flat[1, :12] = [4.0, .25, -.25, .75, 1.25, 1.75, 2.5, -3.5, 5.0, 6.5, 7.75, -0.0]  # scale 1: every tie
        flat[1, 12:] = 0.1
        flat[2] = 2.0 ** -126 * np.linspace(-1, 1, 32)     # shared exponent at its floor
        flat[3] = 2.0 ** -133 * np.arange(32)              # subnormal amax
        flat[4] = 3.0e38 * np.linspace(-1, 1, 32)          # near fp32's top
        flat[5] = np.where(np.arange(32) == 5, 448.0, 475.0 * np.linspace(0, 1, 32))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(1, 32), (8, 64), (1, 8224), (3, 96), (129, 128), (1027, 64), (33, 7168)])
def test_vectors_match_the_exact_codec(rows, D, dtype):
    rng = np.random.default_rng(rows * 1000 + D)
    x = _values(rng, rows, D, dtype)
    codes, bscale = api.mxfp4_quantize(x.cuda())
    c, s = codecs.mx_fp4_quantize(to_f64(x))
    assert np.array_equal(bscale.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), codecs.pack_nibbles(c))
    back = api.mxfp4_dequantize(codes, bscale, dtype=torch.float32)
    assert np.array_equal(to_f64(back), codecs.mx_fp4_decode(c, s).astype(np.float32).astype(np.float64))
    back16 = api.mxfp4_dequantize(codes, bscale)  # bf16: one rounding of the fp32 value (its subnormals)
    assert torch.equal(back16, back.to(torch.bfloat16))


def test_vector_decode_covers_every_byte_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()              # [256, 256]
    bscale = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 16).contiguous().cuda()
    out = to_f64(api.mxfp4_dequantize(codes, bscale, dtype=torch.float32))
    c = codecs.unpack_nibbles(codes.cpu().numpy())
    with np.errstate(over="ignore"):
        ref = codecs.mx_fp4_decode(c, bscale.cpu().numpy()).astype(np.float32).astype(np.float64)
    assert np.array_equal(out, ref, equal_nan=True)
    # bf16: the exact value rounded once, at bf16's range (subnormals, infinity)
    out16 = api.mxfp4_dequantize(codes, bscale)
    with np.errstate(over="ignore"):
        exact = torch.from_numpy(codecs.mx_fp4_decode(c, bscale.cpu().numpy()).astype(np.float32)).to(torch.bfloat16)
    assert np.array_equal(to_f64(out16), to_f64(exact), equal_nan=True)


def test_row_decode_covers_every_byte_and_scale():
    """Rows with one scale code in all blocks and every byte value, decoded to both types."""
    p = np.zeros((256, 176), dtype=np.uint8)
    p[:, :160] = np.arange(160)[None]
    p[128:, :160] = 96 + np.arange(160)[None]
    e = np.concatenate([np.arange(0, 256, 2), np.arange(1, 256, 2)])
    p[:, 160:168] = e[:, None]
    rope = p[:, 32:96]
    rope[(rope & 0x7F) == 0x7F] = 0                    # the quantiser writes no NaN code
    cache = torch.from_numpy(p).cuda()
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(kv4.decode_rows(p).astype(np.float32))
    assert np.array_equal(to_f64(api.kv_dequantize_fp4(cache, dtype=torch.float32)), to_f64(ref), equal_nan=True)
    assert np.array_equal(to_f64(api.kv_dequantize_fp4(cache)), to_f64(ref.to(torch.bfloat16)), equal_nan=True)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_blocks(bad):
    x = torch.ones(2, 96)
    x[0, 40] = bad
    codes, bscale = api.mxfp4_quantize(x.cuda())
    assert bscale.cpu().tolist() == [[125, 255, 125], [125, 125, 125]]
    assert not codes[0, 16:32].any()
    back = api.mxfp4_dequantize(codes, bscale, dtype=torch.float32).cpu()
    assert back[0, 32:64].isnan().all() and (back[0, :32] == 1).all() and (back[1] == 1).all()
    rows = torch.ones(2, 256)
    rows[1, 64 + 35] = bad
    p = api.kv_quantize_fp4(rows.cuda())
    assert np.array_equal(p.cpu().numpy(), kv4.quantize_rows_f64(rows.numpy()))
    v = api.kv_dequantize_fp4(p).float().cpu()
    assert v[1, 96:128].isnan().all() and (v[1, :96] == 1).all() and (v[1, 128:] == 1).all() and (v[0] == 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 2053])
def test_rows_match_the_exact_definition(n, dtype):
    rng = np.random.default_rng(n)
    x = _values(rng, n, 256, dtype)
    p = api.kv_quantize_fp4(x.cuda())
    ref = kv4.quantize_rows_f64(to_f64(x))
    assert np.array_equal(p.cpu().numpy(), ref)
    v = to_f64(api.kv_dequantize_fp4(p, dtype=torch.float32))
    assert np.array_equal(v, kv4.decode_rows(ref).astype(np.float32).astype(np.float64))


def test_rows_scatter_and_gather():
    rng = np.random.default_rng(5)
    n, cap = 77, 200
    x = _values(rng, n, 256, "bf16").cuda()
    dst = torch.from_numpy(rng.permutation(cap)[:n].astype(np.int64))
    dst[3] = -1
    dst[50] = cap + 5                      # out of range: flagged and left out
    before = torch.from_numpy(rng.integers(0, 256, (cap, 176), dtype=np.uint8))
    cache, st = before.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    api.kv_quantize_fp4(x, cache, dst=dst.cuda(), dev_status=st)
    assert int(st.item()) == _lib.DEV_BAD_INDEX
    ref = before.numpy().copy()
    rows = kv4.quantize_rows_f64(to_f64(x))
    for i, d in enumerate(dst.tolist()):
        if 0 <= d < cap:
            ref[d] = rows[i]
    assert np.array_equal(cache.cpu().numpy(), ref)   # rows that were not named are untouched
    st.zero_()
    good = [d for d in dst.tolist() if 0 <= d < cap]
    src = torch.tensor(good + [good[0], -7, cap], dtype=torch.int64).cuda()   # a row twice, none, out of range
    v = to_f64(api.kv_dequantize_fp4(cache, src=src, dev_status=st))
    assert int(st.item()) == _lib.DEV_BAD_INDEX
    k = len(good)
    dec = kv4.decode_rows(ref[good])
    exact = torch.from_numpy(dec).to(torch.float32).to(torch.bfloat16)
    assert np.array_equal(v[:k], to_f64(exact)) and np.array_equal(v[k], v[0])
    assert not v[k + 1:].any()


def test_graph_capture_and_side_stream():
    """The calls run on the current stream and replay from a graph on new inputs."""
    rng = np.random.default_rng(9)
    x = _values(rng, 40, 256, "bf16").cuda()
    cache = torch.zeros(40, 176, dtype=torch.uint8, device="cuda")
    vals = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.kv_quantize_fp4(x, cache)
        api.kv_dequantize_fp4(cache, vals)
        codes, bscale = api.mxfp4_quantize(x)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.kv_quantize_fp4(x, cache)
        api.kv_dequantize_fp4(cache, vals)
        api.mxfp4_quantize(x, codes, bscale)
    y = _values(np.random.default_rng(10), 40, 256, "bf16")
    x.copy_(y)
    g.replay()
    ref = kv4.quantize_rows_f64(to_f64(y))
    assert np.array_equal(cache.cpu().numpy(), ref)
    c, sc = codecs.mx_fp4_quantize(to_f64(y))
    assert np.array_equal(codes.cpu().numpy(), codecs.pack_nibbles(c)) and np.array_equal(bscale.cpu().numpy(), sc)


def test_empty_calls_and_refusals():
    d = "cuda"
    c, b = api.mxfp4_quantize(torch.empty(0, 64, device=d))
    assert c.shape == (0, 32) and b.shape == (0, 2)
    assert api.kv_quantize_fp4(torch.empty(0, 256, device=d)).shape == (0, 176)
    x = torch.zeros(4, 64, device=d)
    with pytest.raises(ValueError):
        api.mxfp4_quantize(torch.zeros(4, 48, device=d))          # not a multiple of 32
    with pytest.raises(ValueError):
        api.mxfp4_quantize(torch.zeros(4, 128, device=d)[:, :64])  # strided
    with pytest.raises(ValueError):
        api.mxfp4_quantize(x.half())
    with pytest.raises(ValueError):
        api.mxfp4_quantize(x.cpu())
    with pytest.raises(ValueError):
        api.mxfp4_dequantize(torch.zeros(4, 32, dtype=torch.uint8, device=d),
                             torch.zeros(4, 1, dtype=torch.uint8, device=d))
    rows = torch.zeros(4, 256, device=d)
    with pytest.raises(ValueError):
        api.kv_quantize_fp4(rows, torch.zeros(4, 336, dtype=torch.uint8, device=d))
    with pytest.raises(ValueError):
        api.kv_quantize_fp4(rows, dst=torch.arange(4, device=d))
    with pytest.raises(CskvError):
        api.kv_quantize_fp4(rows, torch.zeros(3, 176, dtype=torch.uint8, device=d))  # fewer rows than n
    with pytest.raises(ValueError):
        api.kv_dequantize_fp4(torch.zeros(4, 176, dtype=torch.uint8, device=d), src=torch.zeros(2, device=d))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_rows_are_the_rows_of_small_calls(dtype):
    # more rows than one pass of the grid takes (a ragged end too): the same bytes as calls of 1000
    # rows, with and without lists, and back
    n = 151_559
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(n, 256, device="cuda", generator=g).to(dtype)
    x[n - 1, 7] = float("inf")
    small = torch.cat([api.kv_quantize_fp4(x[i:i + 1000].contiguous()) for i in range(0, n, 1000)])
    whole = api.kv_quantize_fp4(x)
    assert torch.equal(whole, small)
    perm = torch.randperm(n, device="cuda", generator=g)
    dst = torch.where(perm % 7 == 3, torch.full_like(perm, -1), perm)
    cache = torch.full((n, 176), 0xAB, dtype=torch.uint8, device="cuda")
    api.kv_quantize_fp4(x, cache, dst=dst)
    kept = dst >= 0
    want = torch.full_like(cache, 0xAB)
    want[dst[kept]] = small[kept]
    assert torch.equal(cache, want)
    back = api.kv_dequantize_fp4(whole, dtype=dtype)
    parts = torch.cat([api.kv_dequantize_fp4(small[i:i + 1000].contiguous(), dtype=dtype) for i in range(0, n, 1000)])
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(back.view(bits), parts.view(bits))
    listed = api.kv_dequantize_fp4(whole, src=dst, dtype=dtype)
    assert torch.equal(listed[kept].view(bits), parts[dst[kept]].view(bits))
    assert torch.count_nonzero(listed[~kept]) == 0
