"""hybrid_decode_attn over 4-bit main-KV rows (CSKV_ATTN_KV_FP4) against attention in float64 over
the same rows decoded exactly (oracle/kv4.py), element by element.

Bounds, before any run.  Decoded rows and bf16 queries are exact in the products, so with
A = sum_r p_r |V_r| (an element's attention over |V|):
* a logit is a sum of 128 exact products in fp32: at most 128 2^-24 sum|q k| scale = dl away (its
  exponential by a factor e^dl), 2 dl A in the quotient;
* P is rounded to bf16 for the product (2^-8 relative; tensor cores only), its sum is not: 2^-8 A;
* accumulation, exponentials and the division in fp32 over R rows: (R + 8) 2^-23 A;
* the output's own rounding: bf16 2^-8 |o|, fp32 2^-24 |o|.
lse: dl + (R + 8) 2^-23 + 2^-22 (1 + |lse|)."""

import math

import numpy as np
import pytest
import torch

from oracle import kv4

from compressed_sparse_kv_compress_b200 import CskvError, _lib, api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    """Sequences of `lens` tokens, `counts` queries each (at their last positions)."""

    def __init__(self, mode, lens, counts, H, k=0, W=128, sink=True, dtype="bf16", seed=0, spread=1.0, skip=0.0):
        self.mode, self.H, self.k, self.W, self.dtype = mode, H, k, W, dtype
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        ratio = 4 if mode == api.CSA else 128
        ent = [-(-n // ratio) for n in lens]
        raw = [min(n, W + c) for n, c in zip(lens, counts)]
        csum = lambda v: np.concatenate([[0], np.cumsum(v)]).astype(np.int64)  # noqa: E731
        self.off, self.raw_off = csum(ent), csum(raw)
        self.t0 = np.array([n - r for n, r in zip(lens, raw)], dtype=np.int64)
        rows = torch.randn(max(1, sum(ent)), 256, generator=g) * torch.exp2(spread * torch.randn(max(1, sum(ent)), 1, generator=g))
        self.cache = torch.from_numpy(kv4.quantize_rows_f64(rows.double().numpy()))
        self.raw = torch.randn(max(1, sum(raw)), 256, generator=g).to(DT[dtype])
        self.q_seq = np.repeat(np.arange(len(lens)), counts).astype(np.int32)
        self.q_pos = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, counts)]).astype(np.int64)
        T = self.T = len(self.q_pos)
        self.q = (torch.randn(T, H, 128, generator=g)).to(DT[dtype])
        self.sink = torch.randn(H, generator=g) if sink else None
        self.most = max([0] + [n // ratio for n in lens])
        self.idx = None
        if mode == api.CSA:
            self.idx = np.full((T, k), -1, dtype=np.int32)
            for t in range(T):
                v = int(self.q_pos[t] + 1) // 4
                e = np.sort(rng.permutation(v)[:k])
                e = np.where(rng.random(len(e)) < skip, -1, e)      # holes inside the list
                self.idx[t, :len(e)] = e

    def dev(self):
        c = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return dict(q=self.q.cuda(), cache=self.cache.cuda(), off=c(self.off), raw=self.raw.cuda(),
                    raw_off=c(self.raw_off), t0=c(self.t0), q_seq=c(self.q_seq), q_pos=c(self.q_pos),
                    idx=None if self.idx is None else c(self.idx), sink=None if self.sink is None else self.sink.cuda())

    def run(self, out_dtype, d=None, out=None, lse=None, ws=None, st=None):
        d = d or self.dev()
        out = torch.full((self.T, self.H, 128), 7.0, dtype=out_dtype, device="cuda") if out is None else out
        lse = torch.full((self.T, self.H), 7.0, device="cuda") if lse is None else lse
        ws = api.attn_workspace(self.mode, self.T, self.H, self.k, self.W, self.most) if ws is None else ws
        st = torch.zeros(1, dtype=torch.int32, device="cuda") if st is None else st
        api.hybrid_decode_attn(self.mode, d["q"], d["cache"], d["off"], d["raw"], d["raw_off"], d["q_seq"],
                               d["q_pos"], out, ws, window=self.W, idx=d["idx"], raw_tok0=d["t0"], sink=d["sink"],
                               lse=lse, max_entries=self.most, kv_fp4=True, dev_status=st)
        return out, lse, st

    def check(self, out, lse, skip_queries=()):
        dec = kv4.decode_rows(self.cache.numpy())
        raw = self.raw.double().numpy()
        o, ls = out.double().cpu().numpy(), lse.double().cpu().numpy()
        scale = 1 / math.sqrt(128)
        tc = self.dtype == "bf16"
        half = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
        for t in range(self.T):
            if t in skip_queries:
                continue
            b, p = int(self.q_seq[t]), int(self.q_pos[t])
            if self.mode == api.CSA:
                e = self.idx[t][self.idx[t] >= 0].astype(np.int64)
            else:
                e = np.arange((p + 1) // 128)
            tok = np.arange(max(0, p - self.W + 1), p + 1) if self.W else np.arange(0)
            kv = np.concatenate([dec[self.off[b] + e], raw[self.raw_off[b] + tok - self.t0[b]]])
            q = self.q[t].double().numpy()
            lg = scale * q @ kv[:, :128].T
            dl = (128 * 2.0 ** -24 * scale * np.abs(q) @ np.abs(kv[:, :128]).T).max(-1) if len(kv) else np.zeros(self.H)
            s = np.full(self.H, -np.inf) if self.sink is None else self.sink.double().numpy()
            M = np.maximum(lg.max(-1) if len(kv) else -np.inf, s)
            M0 = np.where(np.isinf(M), 0, M)
            w = np.exp(lg - M0[:, None])
            L = w.sum(-1) + np.exp(s - M0)
            pr = w / np.where(L > 0, L, 1)[:, None]
            ref, A = pr @ kv[:, 128:], pr @ np.abs(kv[:, 128:])
            R = len(kv)
            tol = (2 * dl[:, None] + (2.0 ** -8 if tc else 0) + (R + 8) * 2.0 ** -23) * A
            tol = tol + half * (np.abs(ref) + tol) + 1e-30
            d = np.abs(o[t] - ref)
            assert np.all(d <= tol), (t, float(d.max()), float((d / tol).max()))
            with np.errstate(divide="ignore"):
                rl = M0 + np.log(L)
            if np.isinf(rl).any():
                assert np.array_equal(np.isinf(rl), ls[t] == -np.inf)
            fin = np.isfinite(rl)
            tl = dl + (R + 8) * 2.0 ** -23 + 2.0 ** -22 * (1 + np.abs(rl))
            dls = np.abs(ls[t][fin] - rl[fin])
            assert np.all(dls <= tl[fin]), (t, dls.max())


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H", [1, 16, 33, 64, 96, 128])
@pytest.mark.parametrize("mode", [api.CSA, api.HCA])
def test_heads_and_outputs(mode, H, out_dtype):
    c = Case(mode, [5000, 900, 130, 3], [2, 1, 1, 1], H, k=200 if mode == api.CSA else 0, seed=H)
    out, lse, st = c.run(out_dtype)
    assert int(st.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [0, 1, 17, 128, 300])
@pytest.mark.parametrize("mode", [api.CSA, api.HCA])
def test_windows_lengths_and_dtypes(mode, W, dtype):
    """Lengths from one token on, chunks that mix compressed and window rows, no sink."""
    lens = [1, 2, 127, 128, 129, 511, 4097]
    c = Case(mode, lens, [1] * len(lens), 16, k=111 if mode == api.CSA else 0, W=W, sink=False, dtype=dtype, seed=W)
    out, lse, st = c.run(torch.float32 if dtype == "f32" else torch.bfloat16)
    assert int(st.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("T,k", [(1, 1024), (40, 512), (149, 1024), (300, 130), (400, 16)])
def test_many_queries_and_splits(T, k):
    """One query split over the SMs up to several queries a CTA (the persistent loop)."""
    c = Case(api.CSA, [6000], [T], 64, k=k, seed=T)
    out, lse, st = c.run(torch.bfloat16)
    assert int(st.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("T,n", [(1, 300000), (3, 70000), (160, 20000)])
def test_dense_lengths(T, n):
    c = Case(api.HCA, [n], [T], 128, seed=n)
    out, lse, st = c.run(torch.bfloat16)
    assert int(st.item()) == 0
    c.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sink", [False, True])
def test_rows_that_masks_leave_empty(sink, dtype):
    """Holes in the selection, queries with no row at all (output 0, lse the sink's or -inf), and
    wide magnitudes, whose maximum moves between chunks."""
    c = Case(api.CSA, [9000, 700], [30, 3], 64, k=500, W=0, sink=sink, seed=11, spread=3.0, skip=0.4, dtype=dtype)
    c.idx[4] = -1
    c.idx[7, :400] = -1          # whole chunks empty first
    c.idx[8, 100:] = -1
    c.idx[31] = -1
    out, lse, st = c.run(torch.float32)
    assert int(st.item()) == 0
    c.check(out, lse)
    assert not out[4].any() and not out[31].any()
    if not sink:
        assert (lse[4] == -math.inf).all()


def test_masked_entries_may_hold_anything():
    """NaN scales in entries that no query selects, and bytes after the last visible entry."""
    c = Case(api.CSA, [4000], [3], 64, k=64, seed=2)
    used = np.unique(c.idx[c.idx >= 0])
    free = np.setdiff1d(np.arange(len(c.cache)), used)
    c.cache[free] = 255
    out, lse, st = c.run(torch.bfloat16)
    assert int(st.item()) == 0 and out.isfinite().all()
    c.check(out, lse)
    h = Case(api.HCA, [1000], [1], 64, seed=3)   # 7 visible entries of 8
    h.cache[7] = 255
    out, lse, st = h.run(torch.bfloat16)
    assert int(st.item()) == 0 and out.isfinite().all()
    h.check(out, lse)


def test_a_nan_entry_that_is_attended_shows():
    c = Case(api.CSA, [4000], [2], 64, k=64, seed=4)
    c.cache[c.idx[1, 5], 160] = 0xFF
    c.idx[0] = np.where(c.idx[0] == c.idx[1, 5], -1, c.idx[0])
    out, lse, _ = c.run(torch.bfloat16)
    assert out[0].isfinite().all() and out[1].isnan().all()
    c.check(out, lse, skip_queries=(1,))


def test_scales_over_the_whole_range():
    """Blocks with every scale code, tiny to huge, decode as the exact values (one-row attention
    returns V itself)."""
    c = Case(api.CSA, [1024], [1], 1, k=1, W=0, sink=False, seed=5)
    row = c.cache[3].clone()
    for e in list(range(0, 4)) + [60, 126, 127, 134, 135, 136, 200, 250, 251]:
        c.cache[3] = row
        c.cache[3, 160:164] = 0          # K: tiny, so the logit is finite
        c.cache[3, 164:168] = e
        c.idx[:] = 3
        out, lse, st = c.run(torch.float32)
        want = kv4.decode_rows(c.cache[3:4].numpy())[0, 128:]
        got = out[0, 0].double().cpu().numpy()
        # bf16's subnormals hold 2^-133 steps; fp32 sums of one product are exact
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -134, 2.0 ** -22 * np.abs(want))), e


def test_bad_indices_are_flagged_and_left_out():
    c = Case(api.CSA, [4000, 800], [2, 1], 16, k=40, seed=6)
    d = c.dev()
    good = c.idx.copy()
    c.idx[0, 3], c.idx[2, 39] = 1000, 200          # not yet complete at those positions
    d["idx"] = torch.from_numpy(c.idx.copy()).cuda()
    out, lse, st = c.run(torch.bfloat16, d)
    assert int(st.item()) == _lib.DEV_BAD_INDEX
    good[0, 3] = good[2, 39] = -1
    c.idx = good
    c.check(out, lse)
    d = c.dev()
    d["q_seq"][1] = 7                               # no such sequence: that query gets zeros
    out, lse, st = c.run(torch.bfloat16, d)
    assert int(st.item()) == _lib.DEV_BAD_INDEX and not out[1].any()
    c.check(out, lse, skip_queries=(1,))


def test_repeats_are_bitwise_equal_and_graphs_replay():
    """No atomics, so the same call gives the same bits; captured graphs replay on new inputs, two
    graphs sharing one workspace in stream order."""
    c = Case(api.CSA, [20000], [5], 64, k=1024, seed=8)
    h = Case(api.HCA, [200000], [2], 64, seed=9)
    d, dh = c.dev(), h.dev()
    a = c.run(torch.bfloat16, d)[0]
    for _ in range(5):
        assert torch.equal(a, c.run(torch.bfloat16, d)[0])
    ws = torch.empty(max(api.attn_workspace_size(api.CSA, 5, 64, 1024, 128, 0),
                         api.attn_workspace_size(api.HCA, 2, 64, 0, 128, h.most)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    oc, lc = torch.empty_like(a), torch.empty(5, 64, device="cuda")
    oh, lh = torch.empty(2, 64, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 64, device="cuda")
    h.run(torch.bfloat16, dh)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        c.run(torch.bfloat16, d, oc, lc, ws, st)
    with torch.cuda.graph(g2):
        h.run(torch.bfloat16, dh, oh, lh, ws, st)
    for seed in (21, 22):
        c2 = Case(api.CSA, [20000], [5], 64, k=1024, seed=seed)
        h2 = Case(api.HCA, [200000], [2], 64, seed=seed)
        for dst, src in ((d, c2.dev()), (dh, h2.dev())):
            for key, t in dst.items():
                if t is not None:
                    t.copy_(src[key])
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        c2.check(oc, lc)
        h2.check(oh, lh)


def test_plain_rows_with_bf16_output():
    """CSKV_ATTN_OUT_BF16 without 4-bit rows: the fp32 result rounded once."""
    for T, H, dtype in ((2, 64, "bf16"), (3, 16, "f32"), (1, 128, "bf16")):
        g = torch.Generator().manual_seed(T)
        kv = torch.randn(300, 256, generator=g).to(DT[dtype]).cuda()
        q = torch.randn(T, H, 128, generator=g).to(DT[dtype]).cuda()
        off = torch.tensor([0, 300], device="cuda")
        pos = torch.arange(38400 - T, 38400, device="cuda")
        raw = torch.randn(T + 128, 256, generator=g).to(DT[dtype]).cuda()
        args = (q, kv, off, raw, torch.tensor([0, T + 128], device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda"), pos)
        ws = api.attn_workspace(api.HCA, T, H, 0, 128, 300)
        kw = dict(window=128, raw_tok0=torch.tensor([38400 - T - 128], device="cuda"), max_entries=300)
        o32, o16 = torch.empty(T, H, 128, device="cuda"), torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
        api.hybrid_decode_attn(api.HCA, *args, o32, ws, **kw)
        api.hybrid_decode_attn(api.HCA, *args, o16, ws, **kw)
        assert torch.equal(o16, o32.to(torch.bfloat16))


def test_refusals():
    c = Case(api.CSA, [400], [1], 16, k=16)
    d = c.dev()
    with pytest.raises(ValueError):
        c.run(torch.float16, d)
    with pytest.raises(ValueError):
        c.run(torch.float32, {**d, "cache": torch.zeros(100, 256, dtype=torch.bfloat16, device="cuda")})
    with pytest.raises(ValueError):
        c.run(torch.float32, {**d, "raw": d["raw"].float()})
    with pytest.raises(CskvError):
        c.run(torch.float32, d, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    lib = _lib.load()
    st = lib.hybrid_decode_attn(api.CSA | _lib.ATTN_KV_FP8 | _lib.ATTN_KV_FP4, 16, 16, 16, 16, 4, 16, 16, None, 4,
                                None, 1.0, 16, 16, 1, 1, 16, 128, _lib.BF16, 0, 16, None, 16, 1 << 20, None, None)
    assert st == _lib.ERR_INVALID_ARG
