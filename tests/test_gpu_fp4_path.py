"""The 4-bit calls together, as a decode step would make them: hidden rows projected to indexer
queries (mxfp4_quantize, mxfp4_matmul), keys and cache rows quantised into their places, the MXFP4
indexer's selection, attention over the 4-bit rows -- each stage against the oracle over the exact
values of the bytes that the stage before it wrote."""

import numpy as np
import pytest
import torch

from oracle import codecs, indexer, kv4

from compressed_sparse_kv_compress_b200 import _lib, api
from helpers import check_selection, to_f64
from test_gpu_attn_kv4 import Case

pytestmark = pytest.mark.gpu


def test_project_index_attend():
    B, Hi, Di, hid, k = 3, 8, 64, 768, 128
    lens = [5001, 2304, 777]
    c = Case(api.CSA, lens, [1] * B, 64, k=k, seed=31)
    d = c.dev()
    n_ent = int(c.off[-1])
    g = torch.Generator().manual_seed(7)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    # cache rows: all but each sequence's last entry in one call, those appended afterwards by row
    rows = torch.randn(n_ent, 256, generator=g).to(torch.bfloat16).cuda()
    last = torch.from_numpy(c.off[1:] - 1).cuda()
    cache = torch.zeros(n_ent, api.KV4_ROW_BYTES, dtype=torch.uint8, device="cuda")
    early = torch.arange(n_ent, device="cuda")
    early[last] = -1
    api.kv_quantize_fp4(rows, cache, dst=early, dev_status=st)
    api.kv_quantize_fp4(rows[last].contiguous(), cache, dst=last, dev_status=st)
    c.cache = cache.cpu()
    assert np.array_equal(c.cache.numpy(), kv4.quantize_rows_f64(to_f64(rows)))
    d["cache"] = cache

    # keys and projected queries in MXFP4
    kc, ke = api.mxfp4_quantize(torch.randn(n_ent, Di, generator=g).cuda())
    w, we = api.mxfp4_quantize((torch.randn(Hi * Di, hid, generator=g) / 28).cuda())
    x, xe = api.mxfp4_quantize(torch.randn(B, hid, generator=g).to(torch.bfloat16).cuda())
    q = api.mxfp4_matmul(x, xe, w, we, dtype=torch.float32, dev_status=st)
    qc, qe = api.mxfp4_quantize(q.view(B, Hi, Di))

    most = max((n // 4) for n in lens)
    idx = torch.empty(B, k, dtype=torch.int32, device="cuda")
    api.lindex_score_topk_mxfp4(qc, qe, kc, ke, d["q_seq"], d["q_pos"], d["off"], idx,
                                api.lindex_workspace(B, k, most), max_entries=most, dev_status=st)
    keys = codecs.mx_fp4_decode(codecs.unpack_nibbles(kc.cpu().numpy()), ke.cpu().numpy())
    qv = codecs.mx_fp4_decode(codecs.unpack_nibbles(qc.cpu().numpy()), qe.cpu().numpy())
    for t in range(B):
        v = indexer.visible_entries(int(c.q_pos[t]), 4)
        s = np.maximum(qv[t] @ keys[c.off[t]:c.off[t] + v].T, 0).sum(0)
        check_selection(idx[t].cpu().numpy(), s, k, f"query {t}")

    c.idx = idx.cpu().numpy()
    d["idx"] = idx
    out, lse, st2 = c.run(torch.bfloat16, d)
    assert int(st.item()) == 0 and int(st2.item()) == 0
    c.check(out, lse)


def test_allocation_free_variant_over_4bit_rows():
    """hybrid_decode_attn_noalloc takes the same flags and gives the same bits."""
    lib = _lib.load()
    for mode, k in ((api.CSA, 300), (api.HCA, 0)):
        c = Case(mode, [40000, 300], [2, 1], 64, k=k, seed=41)
        d = c.dev()
        out, lse, _ = c.run(torch.bfloat16, d)
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        st = lib.hybrid_decode_attn_noalloc(
            mode | _lib.ATTN_KV_FP4 | _lib.ATTN_OUT_BF16, p(d["q"]), p(d["cache"]), p(d["off"]), p(d["idx"]), k,
            p(d["raw"]), p(d["raw_off"]), p(d["t0"]), c.W, p(d["sink"]), 128 ** -0.5, p(d["q_seq"]), p(d["q_pos"]),
            2, c.T, c.H, 128, _lib.BF16, c.most, p(o2), p(l2), None, torch.cuda.current_stream().cuda_stream)
        assert st == _lib.OK
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_two_streams_at_once():
    """The same calls on two streams with workspaces of their own, overlapping on the GPU."""
    cs = [Case(api.CSA, [9000 + 64 * i], [6], 64, k=512, seed=50 + i) for i in range(2)]
    ds = [c.dev() for c in cs]
    ref = [c.run(torch.bfloat16, d)[0] for c, d in zip(cs, ds)]
    a, ae = api.mxfp4_quantize(torch.randn(40, 2048, device="cuda"))
    b, be = api.mxfp4_quantize(torch.randn(1024, 2048, device="cuda"))
    mm = api.mxfp4_matmul(a, ae, b, be)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got, prod = [], []
    for _ in range(20):
        for s, c, d in zip(streams, cs, ds):
            with torch.cuda.stream(s):
                got.append(c.run(torch.bfloat16, d)[0])
                prod.append(api.mxfp4_matmul(a, ae, b, be))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[i % 2]) for i, o in enumerate(got))
    assert all(torch.equal(o, mm) for o in prod)
