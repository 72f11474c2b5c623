"""hybrid_decode_attn over 4-bit rows at its edges: NaN entries that are attended (a block with an infinity
or a NaN reads as NaN, so it has to show in whatever attends to it), and calls that need no workspace."""

import numpy as np
import pytest
import torch

from compressed_sparse_kv_compress_b200 import CskvError, _lib, api
from test_gpu_attn_kv4 import Case

pytestmark = pytest.mark.gpu

NAN_BF16 = torch.tensor(float("nan"), dtype=torch.bfloat16)


def _all_nan(out, lse, t):
    assert bool(out[t].isnan().all()) and bool(lse[t].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("T", [3, 200])
def test_the_only_attended_row_is_nan(T, sink, dtype):
    """Query 1 attends to one row, whose K has a NaN scale; the others' rows are numbers."""
    c = Case(api.CSA, [2000], [T], 64, k=8, W=0, sink=sink, dtype=dtype, seed=3)
    c.idx[c.idx == 7] = -1
    c.idx[1] = -1
    c.idx[1, 2] = 7
    c.cache[7, 160] = 0xFF
    out, lse, _ = c.run(torch.float32)
    _all_nan(out, lse, 1)
    c.check(out, lse, skip_queries=(1,))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_a_split_of_its_own(dtype):
    """1024 selected rows and a window of one token, whose K is NaN: the last split holds that row alone."""
    c = Case(api.CSA, [9000], [1], 64, k=1024, W=1, dtype=dtype, seed=4)
    c.raw[-1, 5] = NAN_BF16
    out, lse, _ = c.run(torch.float32)
    _all_nan(out, lse, 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 160])
def test_nan_rows_before_others(T, dtype):
    """The first 200 rows NaN, the rest numbers; and one NaN row behind 600 numbers."""
    c = Case(api.CSA, [9000], [T], 64, k=700, W=0, sink=False, dtype=dtype, seed=5)
    c.idx[:] = np.arange(700)
    keep = c.cache[:700, 160:164].clone()
    c.cache[:200, 160:164] = 0xFF
    out, lse, _ = c.run(torch.float32)
    for t in range(T):
        _all_nan(out, lse, t)
    c.cache[:700, 160:164] = keep
    c.cache[650, 161] = 0xFF
    out, lse, _ = c.run(torch.float32)
    for t in range(T):
        _all_nan(out, lse, t)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_nan_value_block_shows_in_its_dims_alone(dtype):
    """V dims 32..63 of one attended row: those dims NaN, the others and lse as without it."""
    c = Case(api.CSA, [4000], [2], 64, k=64, dtype=dtype, seed=6)
    ref, ref_lse, _ = c.run(torch.float32)
    e = c.idx[1, 5]
    c.idx[0] = np.where(c.idx[0] == e, -1, c.idx[0])
    c.cache[e, 165] = 0xFF
    out, lse, _ = c.run(torch.float32)
    assert bool(out[1, :, 32:64].isnan().all())
    assert torch.equal(out[1, :, :32], ref[1, :, :32]) and torch.equal(out[1, :, 64:], ref[1, :, 64:])
    assert torch.equal(lse[1], ref_lse[1]) and bool(out[0].isfinite().all())


@pytest.mark.parametrize("mode,k", [(api.CSA, 1024), (api.HCA, 0)])
@pytest.mark.parametrize("T", [1, 70, 80, 400])
def test_many_queries_without_a_workspace(mode, k, T):
    """Queries that are not split write their outputs themselves: no workspace, and the allocation-free
    variant takes any number of them.  Split queries: refused without one, and the variant's own fits."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(mode, [200000], [T], 128, k=k, seed=7)
    d = c.dev()
    out, lse, _ = c.run(torch.bfloat16, d)
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    lib = _lib.load()

    def call(fn, *ws):
        return fn(mode | _lib.ATTN_KV_FP4 | _lib.ATTN_OUT_BF16, p(d["q"]), p(d["cache"]), p(d["off"]), p(d["idx"]), k,
                  p(d["raw"]), p(d["raw_off"]), p(d["t0"]), c.W, p(d["sink"]), 128 ** -0.5, p(d["q_seq"]), p(d["q_pos"]),
                  1, T, 128, 128, _lib.BF16, c.most, p(o2), p(l2), *ws, None, torch.cuda.current_stream().cuda_stream)

    assert call(lib.hybrid_decode_attn_noalloc) == _lib.OK
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert call(lib.hybrid_decode_attn, None, 0) == (_lib.OK if 2 * T > sms else _lib.ERR_WORKSPACE)

    def without():
        o2.fill_(7.0), l2.fill_(7.0)
        api.hybrid_decode_attn(mode, d["q"], d["cache"], d["off"], d["raw"], d["raw_off"], d["q_seq"], d["q_pos"], o2, None,
                               window=c.W, idx=d["idx"], raw_tok0=d["t0"], sink=d["sink"], lse=l2, max_entries=c.most,
                               kv_fp4=True)

    if 2 * T > sms:
        without()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    else:
        with pytest.raises(CskvError):
            without()
