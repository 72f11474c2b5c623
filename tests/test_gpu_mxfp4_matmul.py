"""mxfp4_matmul against the product of the exactly decoded values in float64.

Bounds, before any run: products of E2M1 values and power-of-two scales are exact, so an output is
off by the accumulation alone.  A tensor core adds K = 64 products a step to an fp32 accumulator;
counting every one of the K additions as rounded (or cut) to 2^-23 of sum_k |a b| gives
K 2^-23 sum|a b|; a bf16 output adds 2^-8 |out|, an fp32 one 2^-24."""

import numpy as np
import pytest
import torch

from oracle import codecs

from compressed_sparse_kv_compress_b200 import CskvError, api
from helpers import to_f64

pytestmark = pytest.mark.gpu


def _mat(rng, rows, K, spread):
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-spread, spread + 1, (rows, K // 32)).repeat(32, 1))
    c, s = codecs.mx_fp4_quantize(x)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return t(codecs.pack_nibbles(c)), t(s), codecs.mx_fp4_decode(c, s)


def _check(out, a, b):
    K = a.shape[1]
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    tol = K * 2.0 ** -23 * mag
    tol = tol + half * (np.abs(ref) + tol)
    d = np.abs(to_f64(out) - ref)
    assert np.all(d <= tol), (float(d.max()), float((d / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 512, 4096), (7, 129, 96), (16, 128, 256), (17, 300, 2080), (33, 64, 288), (64, 1000, 544),
    (65, 64, 32), (67, 1000, 2080), (128, 192, 256), (129, 193, 512), (200, 40, 1312), (300, 512, 1024),
    (1000, 1001, 160)])
def test_sizes(M, N, K, dtype):
    """Single rows up to several tiles each way; inner lengths that end inside a tile, and scale rows
    that are not whole words."""
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, ae, av = _mat(rng, M, K, 3)
    b, be, bv = _mat(rng, N, K, 3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    api.mxfp4_matmul(a, ae, b, be, out, dev_status=st)
    assert int(st.item()) == 0
    _check(out, av, bv)


def test_many_tiles_a_cta():
    """More tiles than SMs: the persistent loop and both accumulators."""
    rng = np.random.default_rng(1)
    a, ae, av = _mat(rng, 2500, 320, 1)
    b, be, bv = _mat(rng, 1800, 320, 1)
    _check(api.mxfp4_matmul(a, ae, b, be, dtype=torch.float32), av, bv)
    _check(api.mxfp4_matmul(a[:20].contiguous(), ae[:20].contiguous(), b, be), av[:20], bv)


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 544), (4000, 4001, 288)])
def test_large_tiles(M, N, K):
    """256-row tiles, several a CTA: sampled rows and columns against float64, every element against
    fp32 (both sums are off by K 2^-23 sum|a b| at most)."""
    g = torch.Generator(device="cuda").manual_seed(M)
    a, ae = api.mxfp4_quantize(torch.randn(M, K, device="cuda", generator=g))
    b, be = api.mxfp4_quantize(torch.randn(N, K, device="cuda", generator=g))
    av, bv = (api.mxfp4_dequantize(x, y, dtype=torch.float32) for x, y in ((a, ae), (b, be)))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.mxfp4_matmul(a, ae, b, be, dtype=torch.float32, dev_status=st)
    assert int(st.item()) == 0
    mag = av.abs() @ bv.abs().T
    assert bool(((out - av @ bv.T).abs() <= 2 * K * 2.0 ** -23 * 1.01 * mag).all())
    rows = torch.tensor([0, 127, 128, 255, 256, M // 2, M - 1], device="cuda")
    _check(out[rows], to_f64(av[rows]), to_f64(bv))
    out16 = api.mxfp4_matmul(a, ae, b, be)
    assert torch.equal(out16, out.to(torch.bfloat16))


def test_each_element_meets_its_scale():
    """One nonzero element a row, at every place of a block row: a wrong scale, row or K order shows."""
    K = 576
    for M in (5, 130):
        a = np.zeros((M, K))
        b = np.zeros((K, K))
        for i in range(M):
            a[i, (37 * i) % K] = 1.5 * 2.0 ** (i % 9)
        np.fill_diagonal(b, [2.0 ** (j % 11 - 5) for j in range(K)])
        ca, sa = codecs.mx_fp4_quantize(a)
        cb, sb = codecs.mx_fp4_quantize(b)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        out = api.mxfp4_matmul(t(codecs.pack_nibbles(ca)), t(sa), t(codecs.pack_nibbles(cb)), t(sb), dtype=torch.float32)
        assert np.array_equal(to_f64(out), codecs.mx_fp4_decode(ca, sa) @ codecs.mx_fp4_decode(cb, sb).T)


def test_scales_that_are_not_aligned_and_nan():
    rng = np.random.default_rng(3)
    a, ae, av = _mat(rng, 70, 256, 2)
    b, be, bv = _mat(rng, 33, 256, 2)
    pad = torch.empty(ae.numel() + 1, dtype=torch.uint8, device="cuda")
    odd = pad[1:].view(70, 8)
    odd.copy_(ae)
    _check(api.mxfp4_matmul(a, odd, b, be, dtype=torch.float32), av, bv)
    ae[4, 3] = 0xFF                                  # a NaN scale: its row, and no other
    out = api.mxfp4_matmul(a, ae, b, be, dtype=torch.float32)
    assert out[4].isnan().all() and out[:4].isfinite().all() and out[5:].isfinite().all()


def test_graph_streams_and_repeats():
    rng = np.random.default_rng(4)
    a, ae, _ = _mat(rng, 260, 1024, 2)
    b, be, bv = _mat(rng, 700, 1024, 2)
    ref = api.mxfp4_matmul(a, ae, b, be)
    for _ in range(5):
        assert torch.equal(ref, api.mxfp4_matmul(a, ae, b, be))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2 = api.mxfp4_matmul(a, ae, b, be)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(ref, o2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.mxfp4_matmul(a, ae, b, be, o2)
    a2, ae2, av2 = _mat(rng, 260, 1024, 2)
    a.copy_(a2)
    ae.copy_(ae2)
    g.replay()
    torch.cuda.synchronize()
    _check(o2, av2, bv)


def test_projection_chain_feeds_the_indexer():
    """Hidden rows -> quantise -> product with 4-bit weights -> quantise: the indexer's query vectors,
    which equal the quantised exact product wherever that is not within the product's error of a
    rounding border."""
    g = torch.Generator().manual_seed(6)
    T, Hi, Di, hid = 9, 8, 64, 1024
    x = torch.randn(T, hid, generator=g).to(torch.bfloat16).cuda()
    wq = (torch.randn(Hi * Di, hid, generator=g) / 32).cuda()
    w, we = api.mxfp4_quantize(wq)
    c, e = api.mxfp4_quantize(x)
    q = api.mxfp4_matmul(c, e, w, we, dtype=torch.float32)
    qc, qe = api.mxfp4_quantize(q.view(T, Hi, Di))
    assert qc.shape == (T, Hi, Di // 2) and qe.shape == (T, Hi, Di // 32)
    rc, rs = codecs.mx_fp4_quantize(to_f64(q).reshape(T, Hi, Di))
    assert np.array_equal(qc.cpu().numpy(), codecs.pack_nibbles(rc)) and np.array_equal(qe.cpu().numpy(), rs)


def test_empty_and_refusals():
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert api.mxfp4_matmul(z(0, 32), z(0, 2), z(5, 32), z(5, 2)).shape == (0, 5)
    assert api.mxfp4_matmul(z(3, 32), z(3, 2), z(0, 32), z(0, 2)).shape == (3, 0)
    with pytest.raises(ValueError):
        api.mxfp4_matmul(z(3, 32), z(3, 2), z(4, 48), z(4, 3))   # inner lengths differ
    with pytest.raises(ValueError):
        api.mxfp4_matmul(z(3, 32), z(3, 1), z(4, 32), z(4, 2))
    with pytest.raises(ValueError):
        api.mxfp4_matmul(z(3, 64)[:, :32], z(3, 2), z(4, 32), z(4, 2))
    with pytest.raises(ValueError):
        api.mxfp4_matmul(z(3, 32), z(3, 2), z(4, 32), z(4, 2), torch.empty(3, 4, dtype=torch.float16, device="cuda"))
    with pytest.raises(CskvError):
        api.mxfp4_matmul(z(3, 8), z(3, 0), z(4, 8), z(4, 0))     # half a block


@pytest.mark.parametrize("at", [0, 1, 2, 3, 4, 8, 16, 32])
@pytest.mark.parametrize("M,N,K", [(5, 70, 96), (40, 200, 2080), (70, 130, 1056), (200, 300, 1152), (130, 200, 1312),
                                   (300, 400, 1280), (513, 200, 1536), (1, 129, 4096)])
def test_every_alignment_of_the_scales(M, N, K, at):
    # scales from `at` bytes into a buffer whose other bytes are NaN scales: one of them in a product
    # would show in every output of its row
    rng = np.random.default_rng(M + K)
    (ac, as_, a), (bc, bs, b) = _mat(rng, M, K, 3), _mat(rng, N, K, 3)

    def shifted(s):
        pad = torch.full((s.numel() + 96,), 0xFF, dtype=torch.uint8, device="cuda")
        v = pad[at:at + s.numel()].view(s.shape)
        v.copy_(s)
        return v

    _check(api.mxfp4_matmul(ac, shifted(as_), bc, shifted(bs), dtype=torch.float32), a, b)
