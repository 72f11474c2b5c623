"""Torch-tensor front end of the cskv C ABI: argument marshalling only.

Every function here turns tensors into pointers, sizes and dtype codes and
calls the C entry point of the same name on the current CUDA stream (or the
one given, on which the outputs that the call allocates are then allocated
too).  All computation happens in the CUDA library.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import ATTN_KV_FP4, ATTN_KV_FP8, ATTN_OUT_BF16, ATTN_PAIRS, BF16, CSA, F32, FP8E4M3, HCA, KV4_ROW_BYTES, KV8_ROW_BYTES, OVERLAP_PREVIOUS  # noqa: F401

_DT = {torch.float32: F32, torch.bfloat16: BF16, torch.uint8: FP8E4M3, torch.float8_e4m3fn: FP8E4M3}


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("cskv expects contiguous tensors")
    return t.data_ptr()


def _dt(t) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _check(fn: str, *specs) -> int:
    """Refuses tensors that `fn` cannot take.  specs: (name, tensor or None, dtypes, shape); all of
    them have to be contiguous and on the current CUDA device (returned), whose stream the call runs on.
    Outputs that the call allocates itself come after it, unchecked: for a few rows a call's time
    is the host's."""
    dev = torch.cuda.current_device()
    for name, t, dtypes, shape in specs:
        if t is None:
            continue
        if t.get_device() != dev:
            raise ValueError(f"{fn}: {name} is on {t.device}, not on the current device cuda:{dev}")
        if t.dtype not in dtypes:
            raise ValueError(f"{fn}: {name} has dtype {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} is not contiguous")
    return dev


_U8 = (torch.uint8,)
_I64 = (torch.int64,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)
_VALUES = (torch.float32, torch.bfloat16)


def _new(fn, shape, dtype, dtypes, device, stream=None):
    """An output of the call's own, which belongs to the stream that the call runs on: memory of another
    stream's may still be in use there."""
    if dtype not in dtypes:
        raise ValueError(f"{fn}: dtype {dtype}")
    if stream is not None:
        with torch.cuda.stream(stream):
            return torch.empty(*shape, dtype=dtype, device=device)
    return torch.empty(*shape, dtype=dtype, device=device)  # the sizes one by one: 1 us less than as a tuple


def _stream(stream, dev=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the handle alone: building torch's stream object costs 3 us a call
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if dev is None else dev)


def csa_compress(x_a, z_a, x_b, z_b, tok_off, ent_off, out, *, max_blocks, bias_a=None, bias_b=None, tok0=None,
                 first_block=None, num_blocks=None, rmsnorm=False, norm_gamma=None, norm_eps=1e-6, k_tok=None,
                 k_codes=None, k_scale=None, overlap_previous=False, dev_status=None, stream=None):
    """rmsnorm: normalise each entry's K and V halves (norm_gamma [256] fp32, K then V; None =
    ones).  k_tok [rows, Di] (rows indexed like x_a): also pool the per-token indexer keys of
    the same entries into k_codes [*, Di] uint8 (E4M3) and k_scale [*] fp32.
    overlap_previous: CSKV_OVERLAP_PREVIOUS (the kernel issued just before this call on the
    stream neither writes its inputs nor reads its outputs; see the C header)."""
    lib = _lib.load()
    k_dt = _dt(k_tok) if k_tok is not None else F32
    Di = int(k_tok.shape[-1]) if k_tok is not None else 0
    st = lib.csa_compress(_ptr(x_a), _ptr(z_a), _ptr(x_b), _ptr(z_b), _ptr(bias_a), _ptr(bias_b), _ptr(tok_off),
                          _ptr(tok0), tok_off.numel() - 1, _ptr(ent_off), _ptr(first_block), _ptr(num_blocks),
                          int(max_blocks), _dt(x_a), _dt(out), _ptr(out), int(bool(rmsnorm)), _ptr(norm_gamma),
                          float(norm_eps), _ptr(k_tok), k_dt, Di, _ptr(k_codes), _ptr(k_scale),
                          OVERLAP_PREVIOUS if overlap_previous else 0, _ptr(dev_status), _stream(stream))
    _lib.check("csa_compress", st)
    return out


def hca_compress(x, z, tok_off, ent_off, out, *, max_blocks, bias=None, tok0=None, first_block=None,
                 num_blocks=None, rmsnorm=False, norm_gamma=None, norm_eps=1e-6, dev_status=None, stream=None):
    lib = _lib.load()
    st = lib.hca_compress(_ptr(x), _ptr(z), _ptr(bias), _ptr(tok_off), _ptr(tok0), tok_off.numel() - 1,
                          _ptr(ent_off), _ptr(first_block), _ptr(num_blocks), int(max_blocks), _dt(x), _dt(out),
                          _ptr(out), int(bool(rmsnorm)), _ptr(norm_gamma), float(norm_eps), _ptr(dev_status),
                          _stream(stream))
    _lib.check("hca_compress", st)
    return out


def rmsnorm_heads(x, out=None, *, gamma=None, eps=1e-6, stream=None):
    """RMSNorm of every 128-dimension row of x ([..., 128], fp32 or bf16) into out (default:
    in place): x / sqrt(mean(x^2) + eps) * gamma."""
    out = x if out is None else out
    lib = _lib.load()
    st = lib.rmsnorm_heads(_ptr(x), _dt(x), x.numel() // x.shape[-1], int(x.shape[-1]), _ptr(gamma), float(eps),
                           _ptr(out), _stream(stream))
    _lib.check("rmsnorm_heads", st)
    return out


def lindex_pool_keys(k_tok, tok_off, ent_off, out_codes, out_scale, *, max_blocks, tok0=None, first_block=None,
                     num_blocks=None, dev_status=None, stream=None):
    """Entry keys of the indexer from per-token keys k_tok [rows, Di] (fp32 or bf16): the mean
    of each 4-token block as E4M3 codes (out_codes [*, Di] uint8) with one fp32 scale per
    entry (out_scale [*])."""
    lib = _lib.load()
    st = lib.lindex_pool_keys(_ptr(k_tok), _dt(k_tok), int(k_tok.shape[-1]), _ptr(tok_off), _ptr(tok0),
                              tok_off.numel() - 1, _ptr(ent_off), _ptr(first_block), _ptr(num_blocks),
                              int(max_blocks), _ptr(out_codes), _ptr(out_scale), _ptr(dev_status), _stream(stream))
    _lib.check("lindex_pool_keys", st)
    return out_codes, out_scale


def lindex_workspace_size(T: int, k: int, max_entries: int) -> int:
    return int(_lib.load().lindex_workspace_size(int(T), int(k), int(max_entries)))


def lindex_workspace_size_scan(T: int, max_entries: int) -> int:
    return int(_lib.load().lindex_workspace_size_scan(int(T), int(max_entries)))


def lindex_workspace(T: int, k: int, max_entries: int, device="cuda", scan_only=False) -> torch.Tensor:
    """A zero-filled workspace; calls hand it back zero-filled.  scan_only: the per-query scan's
    size (many-query calls then skip the tensor-core path)."""
    n = lindex_workspace_size_scan(T, max_entries) if scan_only else lindex_workspace_size(T, k, max_entries)
    return torch.zeros(max(16, n), dtype=torch.uint8, device=device)


def lindex_score_topk(q_idx, k_idx, q_seq, q_pos, ent_off, out_idx, workspace, *, max_entries, q_scale=None,
                      k_scale=None, head_w=None, out_score=None, prefetch_rows=None, dev_status=None, stream=None):
    """prefetch_rows: optional [entries, ...] tensor indexed like k_idx (e.g. the compressed
    CSA cache); the rows of the kept entries are prefetched into L2 (a hint)."""
    T, Hi, Di = q_idx.shape
    lib = _lib.load()
    pf_bytes = 0 if prefetch_rows is None else prefetch_rows[0].numel() * prefetch_rows.element_size()
    st = lib.lindex_score_topk(_ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale), _ptr(head_w), _ptr(q_seq),
                               _ptr(q_pos), _ptr(ent_off), ent_off.numel() - 1, T, Hi, Di, out_idx.shape[1],
                               _dt(q_idx), int(max_entries), _ptr(out_idx), _ptr(out_score), _ptr(prefetch_rows),
                               pf_bytes, _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _ptr(dev_status), _stream(stream))
    _lib.check("lindex_score_topk", st)
    return out_idx


def lindex_score_topk_mxfp4(q_codes, q_bscale, k_codes, k_bscale, q_seq, q_pos, ent_off, out_idx, workspace, *,
                            max_entries, q_scale=None, head_w=None, out_score=None, prefetch_rows=None,
                            dev_status=None, stream=None):
    """MXFP4 indexer vectors: q_codes [T, Hi, Di/2] / k_codes [Nc, Di/2] uint8 (two E2M1 codes a
    byte) with E8M0 block scales q_bscale [T, Hi, Di/32] / k_bscale [Nc, Di/32] uint8."""
    T, Hi, half = q_codes.shape
    lib = _lib.load()
    pf_bytes = 0 if prefetch_rows is None else prefetch_rows[0].numel() * prefetch_rows.element_size()
    st = lib.lindex_score_topk_mxfp4(_ptr(q_codes), _ptr(q_bscale), _ptr(q_scale), _ptr(k_codes), _ptr(k_bscale),
                                     _ptr(head_w), _ptr(q_seq), _ptr(q_pos), _ptr(ent_off), ent_off.numel() - 1, T,
                                     Hi, 2 * half, out_idx.shape[1], int(max_entries), _ptr(out_idx),
                                     _ptr(out_score), _ptr(prefetch_rows), pf_bytes, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                     _stream(stream))
    _lib.check("lindex_score_topk_mxfp4", st)
    return out_idx


def lindex_topk_from_scores(scores, n_valid, out_idx, workspace, *, max_entries, out_score=None, dev_status=None,
                            stream=None):
    T, ld = scores.shape
    lib = _lib.load()
    st = lib.lindex_topk_from_scores(_ptr(scores), ld, _ptr(n_valid), T, out_idx.shape[1], int(max_entries),
                                     _ptr(out_idx), _ptr(out_score), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                     _stream(stream))
    _lib.check("lindex_topk_from_scores", st)
    return out_idx


def attn_workspace_size(mode: int, T: int, H: int, k: int, window: int, max_entries: int) -> int:
    return int(_lib.load().hybrid_attn_workspace_size(int(mode), int(T), int(H), 128, int(k), int(window),
                                                      int(max_entries)))


def attn_workspace(mode, T, H, k, window, max_entries, device="cuda") -> torch.Tensor:
    n = attn_workspace_size(mode, T, H, k, window, max_entries)
    return torch.empty(max(16, n), dtype=torch.uint8, device=device)


def _check_attn_kv4(T, H, d, q, kv_cmp, cmp_off, kv_raw, raw_off, q_seq, q_pos, out, idx, raw_tok0, sink, lse, workspace,
                    dev_status):
    """Refuses what attention over 4-bit rows cannot take: its kernels read every array by the counts and
    types that the C header gives.  A call's time for few queries is the host's, so what fits is seen
    by elements and types first (that all are contiguous, as their pointers are taken); only what does
    not goes through the check that names it."""
    dev, B = torch.cuda.current_device(), cmp_off.numel() - 1
    i64, i32, f32 = torch.int64, torch.int32, torch.float32
    if (q.dtype in _VALUES and out.dtype in _VALUES and kv_raw.dtype is q.dtype and kv_cmp.dtype is torch.uint8
            and out.shape == q.shape and kv_cmp.dim() == 2 and kv_cmp.shape[1] == KV4_ROW_BYTES
            and kv_raw.dim() == 2 and kv_raw.shape[1] == 256
            and cmp_off.dtype is i64 and raw_off.dtype is i64 and q_pos.dtype is i64 and q_seq.dtype is i32
            and raw_off.numel() == B + 1 and q_pos.numel() == T and q_seq.numel() == T
            and q.get_device() == dev and out.get_device() == dev and kv_raw.get_device() == dev
            and kv_cmp.get_device() == dev and cmp_off.get_device() == dev and raw_off.get_device() == dev
            and q_pos.get_device() == dev and q_seq.get_device() == dev
            and (idx is None or idx.dtype is i32 and idx.dim() == 2 and idx.shape[0] == T and idx.get_device() == dev)
            and (raw_tok0 is None or raw_tok0.dtype is i64 and raw_tok0.numel() == B and raw_tok0.get_device() == dev)
            and (sink is None or sink.dtype is f32 and sink.numel() == H and sink.get_device() == dev)
            and (lse is None or lse.dtype is f32 and lse.numel() == T * H and lse.get_device() == dev)
            and (workspace is None or workspace.get_device() == dev)
            and (dev_status is None or dev_status.dtype is i32 and dev_status.get_device() == dev)):
        return
    any_of = lambda t: ((t.dtype,), t.shape) if t is not None else (None, None)  # noqa: E731
    _check("hybrid_decode_attn", ("q", q, _VALUES, (T, H, d)), ("kv_cmp", kv_cmp, _U8, (kv_cmp.shape[0], KV4_ROW_BYTES)),
           ("kv_raw", kv_raw, (q.dtype,), (kv_raw.shape[0], 256)), ("out", out, _VALUES, (T, H, d)),
           ("cmp_off", cmp_off, _I64, (B + 1,)), ("raw_off", raw_off, _I64, (B + 1,)), ("q_seq", q_seq, _I32, (T,)),
           ("q_pos", q_pos, _I64, (T,)), ("idx", idx, _I32, (T, idx.shape[-1]) if idx is not None else None),
           ("raw_tok0", raw_tok0, _I64, (B,)), ("sink", sink, _F32, (H,)), ("lse", lse, _F32, (T, H)),
           ("dev_status", dev_status, _I32, dev_status.shape if dev_status is not None else None),
           ("workspace", workspace, *any_of(workspace)))


def hybrid_decode_attn(mode, q, kv_cmp, cmp_off, kv_raw, raw_off, q_seq, q_pos, out, workspace, *, window,
                       idx=None, raw_tok0=None, sink=None, scale=None, lse=None, max_entries=0, adjacent_pairs=False,
                       kv_fp8=False, kv_fp4=False, dev_status=None, stream=None):
    """adjacent_pairs: CSKV_ATTN_PAIRS (queries 2j, 2j + 1 are one sequence's consecutive
    positions; see the C header).  kv_fp8: CSKV_ATTN_KV_FP8, kv_cmp holds FP8 main-KV rows
    ([entries, 336] uint8, from kv_quantize_fp8).  kv_fp4: CSKV_ATTN_KV_FP4, kv_cmp holds 4-bit
    main-KV rows ([entries, 176] uint8, from kv_quantize_fp4).  out is [T, H, 128] fp32, or bf16
    (CSKV_ATTN_OUT_BF16).  workspace: attn_workspace(...); bf16 queries over 4-bit rows may go without
    (None) when they are more than half of the device's SMs."""
    T, H, d = q.shape
    if adjacent_pairs:
        mode = int(mode) | ATTN_PAIRS
    if kv_fp8:
        mode = int(mode) | ATTN_KV_FP8
    if kv_fp4:
        mode = int(mode) | ATTN_KV_FP4
        _check_attn_kv4(T, H, d, q, kv_cmp, cmp_off, kv_raw, raw_off, q_seq, q_pos, out, idx, raw_tok0, sink, lse,
                        workspace, dev_status)
    if out.dtype == torch.bfloat16:
        mode = int(mode) | ATTN_OUT_BF16
    k = idx.shape[1] if idx is not None else 0
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    lib = _lib.load()
    st = lib.hybrid_decode_attn(int(mode), _ptr(q), _ptr(kv_cmp), _ptr(cmp_off), _ptr(idx), k, _ptr(kv_raw),
                                _ptr(raw_off), _ptr(raw_tok0), int(window), _ptr(sink), scale, _ptr(q_seq),
                                _ptr(q_pos), cmp_off.numel() - 1, T, H, d, _dt(q), int(max_entries), _ptr(out),
                                _ptr(lse), _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))
    _lib.check("hybrid_decode_attn", st)
    return out


def copy_segments(src, src_off, dst_ptrs, lens, stream=None):
    """Scatter segments of the byte buffer `src` (int64 device arrays src_off, lens and
    dst_ptrs = destination addresses) with one kernel: the unpacking half of a staged
    host-to-device copy of a step's new inputs, or a read-back into host memory.  `src` is a
    device tensor or an address from mapped_pointer(); host destinations in dst_ptrs must be
    mapped_pointer() addresses too."""
    lib = _lib.load()
    src_p = src if isinstance(src, int) else _ptr(src)
    st = lib.cskv_copy_segments(src_p, _ptr(src_off), _ptr(dst_ptrs), _ptr(lens), int(src_off.numel()),
                                _stream(stream))
    _lib.check("cskv_copy_segments", st)


def kv_quantize_fp8(rows, out=None, stream=None):
    """FP8 main-KV rows ([n, 336] uint8) from K||V rows [n, 256] (fp32 or bf16, device)."""
    assert rows.dim() == 2 and rows.shape[1] == 256
    n = rows.shape[0]
    if out is None:
        out = _new("kv_quantize_fp8", (n, KV8_ROW_BYTES), torch.uint8, _U8, rows.device, stream)
    lib = _lib.load()
    st = lib.kv_quantize_fp8(_ptr(rows), _dt(rows), n, _ptr(out), _stream(stream))
    _lib.check("kv_quantize_fp8", st)
    return out


def _mxfp4_shapes(fn, lead, D):
    """Shapes of the codes and scales of vectors [*lead, D]."""
    if D < 1 or D % 32:
        raise ValueError(f"{fn}: rows of {D} values; MXFP4 takes a multiple of 32")
    return (*lead, D // 2), (*lead, D // 32)


def mxfp4_quantize(x, codes=None, bscale=None, *, stream=None):
    """MXFP4 form of x [..., D] (fp32 or bf16, D a multiple of 32): (codes [..., D/2] uint8, two
    E2M1 codes a byte, bscale [..., D/32] uint8, one E8M0 scale per 32 values)."""
    *lead, D = x.shape
    cs, bs = _mxfp4_shapes("mxfp4_quantize", lead, D)
    dev = _check("mxfp4_quantize", ("x", x, _VALUES, x.shape), ("codes", codes, _U8, cs), ("bscale", bscale, _U8, bs))
    if codes is None:
        codes = _new("mxfp4_quantize", cs, torch.uint8, _U8, x.device, stream)
    if bscale is None:
        bscale = _new("mxfp4_quantize", bs, torch.uint8, _U8, x.device, stream)
    st = _lib.load().mxfp4_quantize(x.data_ptr(), _DT[x.dtype], x.numel() // D, D, codes.data_ptr(),
                                    bscale.data_ptr(), _stream(stream, dev))
    _lib.check("mxfp4_quantize", st)
    return codes, bscale


def mxfp4_dequantize(codes, bscale, out=None, *, dtype=torch.bfloat16, stream=None):
    """The values [..., D] of MXFP4 codes [..., D/2] with scales [..., D/32], as `dtype` (or out's)."""
    *lead, half = codes.shape
    D = 2 * half
    _, bs = _mxfp4_shapes("mxfp4_dequantize", lead, D)
    dev = _check("mxfp4_dequantize", ("codes", codes, _U8, codes.shape), ("bscale", bscale, _U8, bs),
           ("out", out, _VALUES, (*lead, D)))
    if out is None:
        out = _new("mxfp4_dequantize", (*lead, D), dtype, _VALUES, codes.device, stream)
    st = _lib.load().mxfp4_dequantize(codes.data_ptr(), bscale.data_ptr(), out.numel() // D, D, _DT[out.dtype],
                                      out.data_ptr(), _stream(stream, dev))
    _lib.check("mxfp4_dequantize", st)
    return out


def mxfp4_matmul(a_codes, a_bscale, b_codes, b_bscale, out=None, *, dtype=torch.bfloat16, dev_status=None, stream=None):
    """out [M, N] = a b^T of MXFP4 matrices (mxfp4_quantize): a_codes [M, K/2], a_bscale [M, K/32],
    b_codes [N, K/2], b_bscale [N, K/32]; out fp32 or bf16 (`dtype`, or out's)."""
    (M, half), (N, _) = a_codes.shape, b_codes.shape
    dev = _check("mxfp4_matmul", ("a_codes", a_codes, _U8, (M, half)), ("a_bscale", a_bscale, _U8, (M, half // 16)),
           ("b_codes", b_codes, _U8, (N, half)), ("b_bscale", b_bscale, _U8, (N, half // 16)),
           ("out", out, _VALUES, (M, N)), ("dev_status", dev_status, _I32, (1,)))
    if out is None:
        out = _new("mxfp4_matmul", (M, N), dtype, _VALUES, a_codes.device, stream)
    st = _lib.load().mxfp4_matmul(a_codes.data_ptr(), a_bscale.data_ptr(), b_codes.data_ptr(), b_bscale.data_ptr(),
                                  M, N, 2 * half, _DT[out.dtype], out.data_ptr(), _ptr(dev_status), _stream(stream, dev))
    _lib.check("mxfp4_matmul", st)
    return out


def kv_quantize_fp4(rows, out=None, *, dst=None, dev_status=None, stream=None):
    """4-bit main-KV rows ([cap, 176] uint8) from K||V rows [n, 256] (fp32 or bf16).  dst [n]
    int64: row i goes to out[dst[i]] (negative: left out; no two equal); None: to out[i].  Rows of
    `out` that are not named stay as they were."""
    n = rows.shape[0]
    if out is None and dst is not None:
        raise ValueError("kv_quantize_fp4: dst needs the cache it points into (out)")
    cap = out.shape[0] if out is not None else n
    dev = _check("kv_quantize_fp4", ("rows", rows, _VALUES, (n, 256)), ("out", out, _U8, (cap, KV4_ROW_BYTES)),
           ("dst", dst, _I64, (n,)), ("dev_status", dev_status, _I32, (1,)))
    if out is None:
        out = _new("kv_quantize_fp4", (n, KV4_ROW_BYTES), torch.uint8, _U8, rows.device, stream)
    st = _lib.load().kv_quantize_fp4(rows.data_ptr(), _DT[rows.dtype], n, _ptr(dst), cap, out.data_ptr(),
                                     _ptr(dev_status), _stream(stream, dev))
    _lib.check("kv_quantize_fp4", st)
    return out


def kv_dequantize_fp4(cache, out=None, *, src=None, dtype=torch.bfloat16, dev_status=None, stream=None):
    """K||V values [n, 256] (`dtype`, or out's) of the 4-bit main-KV rows cache [cap, 176]: rows
    src [n] int64 of it (negative: zeros), or its first rows (all of them without `out`)."""
    cap = cache.shape[0]
    n = src.shape[0] if src is not None else out.shape[0] if out is not None else cap
    dev = _check("kv_dequantize_fp4", ("cache", cache, _U8, (cap, KV4_ROW_BYTES)), ("out", out, _VALUES, (n, 256)),
           ("src", src, _I64, (n,)), ("dev_status", dev_status, _I32, (1,)))
    if out is None:
        out = _new("kv_dequantize_fp4", (n, 256), dtype, _VALUES, cache.device, stream)
    st = _lib.load().kv_dequantize_fp4(cache.data_ptr(), _ptr(src), cap, n, _DT[out.dtype], out.data_ptr(),
                                       _ptr(dev_status), _stream(stream, dev))
    _lib.check("kv_dequantize_fp4", st)
    return out


def mapped_pointer(t) -> int:
    """The address at which the current device reaches tensor `t`'s data: its own address for
    device memory, the mapped address for page-locked host memory.  Raises for pageable host
    memory, which the device cannot address."""
    lib = _lib.load()
    out = ctypes.c_void_p()
    st = lib.cskv_mapped_pointer(_ptr(t), ctypes.byref(out))
    _lib.check("cskv_mapped_pointer", st)
    return int(out.value)
