"""hybrid_decode_attn over 4-bit rows where the warps of a CTA drift apart, against attention in float64
element by element (bounds in test_gpu_attn_kv4.py): heads whose maxima grow with every chunk, so that
their 32-head group rescales its output in each, beside groups whose maxima stay."""

import math

import numpy as np
import pytest
import torch

from oracle import kv4

from compressed_sparse_kv_compress_b200 import _lib, api
from test_gpu_attn_kv4 import Case

pytestmark = pytest.mark.gpu

GROW = 9.0  # log2 of a maximum's growth from chunk to chunk (the kernel rescales from 8 on)


def _rising(c, group, levels, raw_level):
    """Logits of the heads 32 group .. 32 group + 31 grow by 2^GROW a level, the others' stay: K dim 64 is
    the row's level, and only those heads' queries look at it."""
    n = len(c.cache)
    rows = np.random.default_rng(group).standard_normal((n, 256))
    rows[:, :128] *= 0.25
    rows[:, 64] = levels
    c.cache = torch.from_numpy(kv4.quantize_rows_f64(rows))
    c.raw[:, :128] *= 0.25
    c.raw[:, 64] = raw_level
    q = 0.25 * c.q.float()
    q[:, :, 64] = 0.0
    q[:, 32 * group:32 * group + 32, 64] = GROW * math.log(2.0) * math.sqrt(128.0)
    c.q = q.to(torch.bfloat16)


@pytest.mark.parametrize("H,group", [(64, 0), (64, 1), (96, 0), (96, 1), (96, 2), (128, 0), (128, 1), (128, 2), (128, 3)])
@pytest.mark.parametrize("T", [1, 160])
def test_groups_of_heads_that_drift_apart(T, H, group):
    """Several chunks a query (T of more than the SMs), and several chunks a split of one query."""
    ent = 1000 if T > 1 else 56832               # 444 chunks: three a split on 148 SMs
    c = Case(api.HCA, [128 * ent], [T], H, W=128 if T > 1 else 0, sink=group % 2 == 0, seed=H + group)
    chunk = np.arange(len(c.cache)) // 128
    if T > 1:
        _rising(c, group, chunk.astype(float), 8.0)
    else:
        _rising(c, group, (chunk % 3).astype(float), 3.0)
    d = c.dev()
    out, lse, st = c.run(torch.float32, d)
    assert int(st.item()) == 0
    c.check(out, lse)
    for _ in range(5):
        again, _, _ = c.run(torch.float32, d)
        assert torch.equal(out, again)


def test_a_whole_prefill_chunk():
    """4096 queries of 64 heads over 1024 selected entries and the window: every element."""
    c = Case(api.CSA, [6000], [4096], 64, k=1024, seed=77)
    d = c.dev()
    out, lse, st = c.run(torch.float32, d)
    assert int(st.item()) == 0
    dec = torch.from_numpy(kv4.decode_rows(c.cache.numpy())).cuda()
    raw = c.raw.double().cuda()
    scale, dev = 1 / math.sqrt(128), "cuda"
    for t0 in range(0, c.T, 64):
        t = torch.arange(t0, t0 + 64, device=dev)
        e = d["idx"][t].long()
        tok = d["q_pos"][t][:, None] - c.W + 1 + torch.arange(c.W, device=dev)
        ok = torch.cat([e >= 0, tok >= 0], 1)
        kv = torch.cat([dec[e.clamp(min=0)], raw[(tok - int(c.t0[0])).clamp(min=0)]], 1)
        q = d["q"][t].double()
        lg = (scale * q @ kv[..., :128].mT).masked_fill(~ok[:, None], -math.inf)
        dl = (128 * 2.0 ** -24 * scale * q.abs() @ kv[..., :128].abs().mT).masked_fill(~ok[:, None], 0).amax(-1)
        full = torch.cat([lg, d["sink"].double()[None, :, None].expand(64, -1, -1)], -1)
        rl = torch.logsumexp(full, -1)
        pr = torch.exp(lg - rl[..., None])
        ref, A = pr @ kv[..., 128:], pr @ kv[..., 128:].abs()
        R = ok.sum(1)[:, None]
        tol = (2 * dl[..., None] + 2.0 ** -8 + (R[..., None] + 8) * 2.0 ** -23) * A
        tol = tol + 2.0 ** -24 * (ref.abs() + tol) + 1e-30
        assert bool(((out[t].double() - ref).abs() <= tol).all()), t0
        tl = dl + (R + 8) * 2.0 ** -23 + 2.0 ** -22 * (1 + rl.abs())
        assert bool(((lse[t].double() - rl).abs() <= tl).all()), t0


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("sink", [False, True])
def test_empty_queries_between_others(H, sink):
    """Dense mode without a window: a CTA's queries (every SMs-th of the list) have rows and none in turn,
    some of them because their sequence does not exist."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 6 * sms + 5
    full = (np.arange(T) // sms) % 2 == 0
    c = Case(api.HCA, [int(n) for n in np.where(full, 128 * (1 + np.arange(T) % 5) + 3, 1 + np.arange(T) % 127)],
             [1] * T, H, W=0, sink=sink, seed=H)
    d = c.dev()
    ref = [c.run(torch.float32, d) for _ in range(8)]
    c.check(ref[0][0], ref[0][1])
    assert all(int(st.item()) == 0 for _, _, st in ref)
    assert all(torch.equal(ref[0][0], o) and torch.equal(ref[0][1], e) for o, e, _ in ref)
    none = np.flatnonzero(~full)
    assert not ref[0][0][none].any()
    d["q_seq"][none[::3]] = T
    out, lse, st = c.run(torch.float32, d)
    assert int(st.item()) == _lib.DEV_BAD_INDEX
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[none[::3]] = False
    assert torch.equal(out, ref[0][0]) and torch.equal(lse[keep], ref[0][1][keep])
