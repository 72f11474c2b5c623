"""The indexer's low-precision projection stage by stage (hidden rows -> mxfp4_quantize -> mxfp4_matmul ->
mxfp4_quantize), each against the definition in float64 over what the stage before it wrote; and bf16
attention outputs over the other row types, which are the fp32 result rounded once."""

import numpy as np
import pytest
import torch

from oracle import codecs

from compressed_sparse_kv_compress_b200 import api
from helpers import to_f64

pytestmark = pytest.mark.gpu


def _values(c, s):
    return codecs.mx_fp4_decode(codecs.unpack_nibbles(c.cpu().numpy()), s.cpu().numpy())


@pytest.mark.parametrize("T,Hi,Di,hid", [(1, 8, 64, 1024), (9, 8, 64, 1024), (3, 8, 64, 768), (70, 16, 128, 2080)])
def test_projected_queries(T, Hi, Di, hid):
    """Products within K 2^-23 sum|a b| (every addition rounded or cut) and the fp32 rounding, then the codes
    of what was written, byte by byte."""
    g = torch.Generator().manual_seed(T + hid)
    x = torch.randn(T, hid, generator=g).to(torch.bfloat16).cuda()
    wt = (torch.randn(Hi * Di, hid, generator=g) / 32).cuda()
    c, e = api.mxfp4_quantize(x)
    w, we = api.mxfp4_quantize(wt)
    for codes, scales, src in ((c, e, x), (w, we, wt)):
        rc, rs = codecs.mx_fp4_quantize(to_f64(src))
        assert np.array_equal(codes.cpu().numpy(), codecs.pack_nibbles(rc)) and np.array_equal(scales.cpu().numpy(), rs)
    q = api.mxfp4_matmul(c, e, w, we, dtype=torch.float32)
    a, b = _values(c, e), _values(w, we)
    ref = a @ b.T
    tol = hid * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    tol = tol + 2.0 ** -24 * (np.abs(ref) + tol)
    assert np.all(np.abs(to_f64(q) - ref) <= tol)
    qc, qe = api.mxfp4_quantize(q.view(T, Hi, Di))
    rc, rs = codecs.mx_fp4_quantize(to_f64(q).reshape(T, Hi, Di))
    assert np.array_equal(qc.cpu().numpy(), codecs.pack_nibbles(rc)) and np.array_equal(qe.cpu().numpy(), rs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("entries", [300, 8192])
@pytest.mark.parametrize("T,H,dtype", [(2, 64, torch.bfloat16), (1, 128, torch.bfloat16), (3, 16, torch.float32)])
def test_bf16_outputs_over_other_rows(T, H, dtype, entries, fp8):
    g = torch.Generator().manual_seed(T + entries)
    n = 128 * entries
    kv = torch.randn(entries, 256, generator=g).to(dtype).cuda()
    kv = api.kv_quantize_fp8(kv) if fp8 else kv
    raw = torch.randn(T + 128, 256, generator=g).to(dtype).cuda()
    q = torch.randn(T, H, 128, generator=g).to(dtype).cuda()
    t = lambda *v: torch.tensor(v, device="cuda")  # noqa: E731
    sink = torch.randn(H, generator=g).cuda()
    outs, lses = [], []
    for od in (torch.float32, torch.bfloat16):
        out, lse = torch.empty(T, H, 128, dtype=od, device="cuda"), torch.empty(T, H, device="cuda")
        api.hybrid_decode_attn(api.HCA, q, kv, t(0, entries), raw, t(0, T + 128), torch.zeros(T, dtype=torch.int32, device="cuda"),
                               torch.arange(n - T, n, device="cuda"), out, api.attn_workspace(api.HCA, T, H, 0, 128, entries),
                               window=128, raw_tok0=t(n - T - 128), sink=sink, lse=lse, max_entries=entries, kv_fp8=fp8)
        outs.append(out), lses.append(lse)
    assert bool(outs[0].isfinite().all())
    assert torch.equal(outs[1], outs[0].to(torch.bfloat16)) and torch.equal(lses[0], lses[1])
