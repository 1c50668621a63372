"""B200 (sm_100a) library for DeepSeek-V4's hybrid attention (CSA + HCA).

This module is the thin Python binding of ``libcsa13.so`` (C ABI declared in
``include/csa.h``).  It only marshals arguments: torch tensors supply device
memory and streams, every computation runs in the library's CUDA kernels.
Importing works without a GPU (the library loads, nothing launches); calling
anything without the built library raises.

Names follow the C ABI: ``csa_compress``, ``csa_quantize``, ``indexer_score``,
``topk_select``, ``sparse_mqa_attn``, ``hca_attn``, ``window_attn``, ``csa_decode``,
``csa_prefill``, ``csa_workspace_size``, ``csa_device_status``, and
``csa_decode_noalloc`` (csa_decode on the library's fixed device scratch, for
callers that cannot allocate).  The grouped-head calls ``paged_append``,
``paged_decode_attn``, ``prompt_attn`` and ``csa_gqa_workspace_size`` take a
``GqaParams``.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass

F32, BF16, FP8_S64, MXFP4 = 0, 1, 2, 3
OP_SPARSE_ATTN, OP_HCA_ATTN, OP_DECODE, OP_PREFILL, OP_WINDOW_ATTN = 0, 1, 2, 3, 4
OP_SHARD_SELECT, OP_SHARD_ATTEND, OP_HCA_SHARD = 5, 6, 7
OP_PAGED_DECODE, OP_PROMPT_ATTN = 8, 9
FLAG_BATCH_INVARIANT = 0x1
FLAG_QI_BF16 = 0x2
FLAG_INDEXER_FP8 = 0x4
FLAG_ROT_PAIRS = 0x8
DEV_BAD_INDEX, DEV_RANGE, DEV_TIMEOUT = 0x1, 0x2, 0x4
NOALLOC_SCRATCH_BYTES = 32 << 20   # CSA_NOALLOC_SCRATCH_BYTES
ERR_WORKSPACE = -4

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa13.so")
_lib = None


class CsaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({strerror(status)})")


class Params(C.Structure):
    """Mirror of ``csa_params``."""
    _fields_ = [("m", C.c_int32), ("window", C.c_int32), ("top_k", C.c_int32),
                ("n_heads", C.c_int32), ("head_dim", C.c_int32), ("idx_heads", C.c_int32),
                ("idx_dim", C.c_int32), ("scale", C.c_float), ("act_fmt", C.c_int32),
                ("kv_fmt", C.c_int32), ("idx_fmt", C.c_int32), ("flags", C.c_uint32)]


def params(m, window, top_k, n_heads, head_dim, idx_heads, idx_dim, scale,
           act_fmt=BF16, kv_fmt=FP8_S64, idx_fmt=MXFP4, flags=0) -> Params:
    return Params(m, window, top_k, n_heads, head_dim, idx_heads, idx_dim, float(scale),
                  act_fmt, kv_fmt, idx_fmt, flags)


class GqaParams(C.Structure):
    """Mirror of ``csa_gqa_params``."""
    _fields_ = [("n_heads", C.c_int32), ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("page_size", C.c_int32), ("window", C.c_int32), ("rot_dim", C.c_int32),
                ("scale", C.c_float), ("act_fmt", C.c_int32), ("cache_fmt", C.c_int32),
                ("flags", C.c_uint32)]


def gqa_params(n_heads, n_kv_heads, head_dim, scale, page_size=16, window=0, rot_dim=0, act_fmt=BF16,
               cache_fmt=BF16, flags=0) -> GqaParams:
    return GqaParams(n_heads, n_kv_heads, head_dim, page_size, window, rot_dim, float(scale), act_fmt,
                     cache_fmt, flags)


EXPORTS = ["csa_compress", "csa_quantize", "indexer_score", "topk_select", "sparse_mqa_attn",
           "hca_attn", "window_attn", "csa_decode", "csa_prefill", "csa_workspace_size",
           "csa_device_status", "csa_strerror", "csa_version", "csa_decode_noalloc",
           "csa_shard_select", "csa_shard_attend", "hca_shard_attend", "attn_merge", "paged_append",
           "paged_decode_attn", "prompt_attn", "csa_gqa_workspace_size"]


def lib():
    """Load libcsa13.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m compressed_sparse_attention_13_b200.build`")
        L = C.CDLL(LIB_PATH)
        P, I32, I64, PP = C.c_void_p, C.c_int32, C.c_int64, C.POINTER(Params)
        L.csa_compress.argtypes = [PP, I32, P, P, P, I64, I32, P, P, P]
        L.csa_quantize.argtypes = [I32, P, I64, I32, P, P, P]
        L.indexer_score.argtypes = [PP, I32, I32, P, P, P, P, P, I64, P, P, I64, P]
        L.topk_select.argtypes = [PP, I32, I32, P, I64, I64, P, P, P]
        L.sparse_mqa_attn.argtypes = [PP, I32, I32, P, P, P, I64, P, P, I64, P, P, P, P, P,
                                      C.c_size_t, P]
        L.hca_attn.argtypes = [PP, I32, I32, P, P, P, I64, P, I64, P, P, P, P, P, C.c_size_t, P]
        L.window_attn.argtypes = [PP, I32, I32, P, P, I64, P, P, P, P, P, C.c_size_t, P]
        L.csa_decode.argtypes = [PP, I32, P, P, P, P, P, P, P, P, I64, P, I64, P, P, P, P, P, P,
                                 C.c_size_t, P]
        L.csa_prefill.argtypes = [PP, I32, I64, I64, P, I64, I64, P, P, P, P, P, P, P, P, P, P,
                                  I64, P, P, P, P, C.c_size_t, P]
        L.csa_decode_noalloc.argtypes = [PP, I32, P, P, P, P, P, P, P, P, I64, P, I64, P, P, P,
                                         P, P, P]
        L.csa_shard_select.argtypes = [PP, I32, P, P, P, P, P, I64, I64, P, P, P, P, C.c_size_t, P]
        L.csa_shard_attend.argtypes = [PP, I32, P, I32, P, P, P, P, I64, I64, P, I64, P, P, P, P, P, P,
                                       C.c_size_t, P]
        L.hca_shard_attend.argtypes = [PP, I32, P, P, P, I64, I64, P, I64, P, P, P, P, P, C.c_size_t, P]
        L.attn_merge.argtypes = [PP, I32, I32, P, P, P, P, P]
        L.csa_workspace_size.restype = C.c_size_t
        L.csa_workspace_size.argtypes = [PP, I32, I32, I64, I64]
        GP = C.POINTER(GqaParams)
        L.paged_append.argtypes = [GP, I32, I64, P, P, P, I64, P, I64, P, I64, P, P, P, P, P, P, P, I64, P, I64, P]
        L.paged_decode_attn.argtypes = [GP, I32, P, I64, P, P, P, P, I64, P, I64, P, P, P, P, C.c_size_t, P]
        L.prompt_attn.argtypes = [GP, I32, P, I64, I64, P, I64, P, I64, I64, P, P, P, P, P, C.c_size_t, P]
        L.csa_gqa_workspace_size.restype = C.c_size_t
        L.csa_gqa_workspace_size.argtypes = [GP, I32, I32, I64, I64]
        L.csa_device_status.argtypes = [P, C.POINTER(C.c_uint32), I32]
        L.csa_strerror.restype = C.c_char_p
        L.csa_strerror.argtypes = [C.c_int]
        L.csa_version.restype = C.c_char_p
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().csa_strerror(status).decode()


def version() -> str:
    return lib().csa_version().decode()


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _s(stream):
    import torch
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _ok(fn, st):
    if st != 0:
        raise CsaError(fn, st)


@dataclass
class Stored:
    """A stored tensor: data plus per-group scales (FP8_S64 / MXFP4)."""
    fmt: int
    data: "object"
    scales: "object" = None


def empty_stored(fmt: int, rows: int, d: int, device="cuda") -> Stored:
    """Allocate (with torch) a [rows][d] tensor in a stored format."""
    import torch
    if fmt == F32:
        return Stored(fmt, torch.empty(rows, d, dtype=torch.float32, device=device))
    if fmt == BF16:
        return Stored(fmt, torch.empty(rows, d, dtype=torch.bfloat16, device=device))
    if fmt == FP8_S64:
        return Stored(fmt, torch.empty(rows, d, dtype=torch.uint8, device=device),
                      torch.empty(rows, d // 64, dtype=torch.float32, device=device))
    if fmt == MXFP4:
        return Stored(fmt, torch.empty(rows, d // 2, dtype=torch.uint8, device=device),
                      torch.empty(rows, d // 32, dtype=torch.uint8, device=device))
    raise ValueError(fmt)


# --------------------------------------------------------------- entry points
def csa_compress(p: Params, d: int, x, z, bias, n_tokens: int, out: Stored, stream=None):
    _ok("csa_compress", lib().csa_compress(C.byref(p), d, _p(x), _p(z), _p(bias), n_tokens,
                                           out.fmt, _p(out.data), _p(out.scales), _s(stream)))


def csa_quantize(src, out: Stored, stream=None):
    d = src.shape[-1]
    rows = src.numel() // d
    _ok("csa_quantize", lib().csa_quantize(out.fmt, _p(src), rows, d, _p(out.data),
                                           _p(out.scales), _s(stream)))


def indexer_score(p: Params, batch: int, n_q: int, qI: Stored, w, kI: Stored, max_blocks: int,
                  q_pos, scores, ld_scores: int, stream=None):
    _ok("indexer_score", lib().indexer_score(
        C.byref(p), batch, n_q, _p(qI.data), _p(qI.scales), _p(w), _p(kI.data), _p(kI.scales),
        max_blocks, _p(q_pos), _p(scores), ld_scores, _s(stream)))


def topk_select(p: Params, batch: int, n_q: int, scores, ld_scores: int, max_blocks: int, q_pos,
                idx, stream=None):
    _ok("topk_select", lib().topk_select(C.byref(p), batch, n_q, _p(scores), ld_scores,
                                         max_blocks, _p(q_pos), _p(idx), _s(stream)))


def csa_workspace_size(p: Params, op: int, batch: int, n_q: int, n_ctx: int) -> int:
    return lib().csa_workspace_size(C.byref(p), op, batch, n_q, n_ctx)


def _ws(ws):
    return (None, 0) if ws is None else (_p(ws), ws.numel() * ws.element_size())


def sparse_mqa_attn(p: Params, batch: int, n_q: int, q, kv: Stored, max_entries: int, idx, raw,
                    n_raw: int, raw_pos0, q_pos, sinks, out, workspace=None, stream=None):
    wp, wb = _ws(workspace)
    _ok("sparse_mqa_attn", lib().sparse_mqa_attn(
        C.byref(p), batch, n_q, _p(q), _p(kv.data), _p(kv.scales), max_entries, _p(idx), _p(raw),
        n_raw, _p(raw_pos0), _p(q_pos), _p(sinks), _p(out), wp, wb, _s(stream)))


def hca_attn(p: Params, batch: int, n_q: int, q, kv: Stored, max_entries: int, raw, n_raw: int,
             raw_pos0, q_pos, sinks, out, workspace=None, stream=None):
    wp, wb = _ws(workspace)
    _ok("hca_attn", lib().hca_attn(
        C.byref(p), batch, n_q, _p(q), _p(kv.data), _p(kv.scales), max_entries, _p(raw), n_raw,
        _p(raw_pos0), _p(q_pos), _p(sinks), _p(out), wp, wb, _s(stream)))


def window_attn(p: Params, batch: int, n_q: int, q, raw, n_raw: int, raw_pos0, q_pos, sinks, out,
                workspace=None, stream=None):
    wp, wb = _ws(workspace)
    _ok("window_attn", lib().window_attn(
        C.byref(p), batch, n_q, _p(q), _p(raw), n_raw, _p(raw_pos0), _p(q_pos), _p(sinks), _p(out),
        wp, wb, _s(stream)))


def csa_decode(p: Params, batch: int, q, qI: Stored, w, kv: Stored, kI: Stored, max_blocks: int,
               raw, n_raw: int, raw_pos0, q_pos, sinks, out, idx_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _ok("csa_decode", lib().csa_decode(
        C.byref(p), batch, _p(q), _p(qI.data), _p(qI.scales), _p(w), _p(kv.data), _p(kv.scales),
        _p(kI.data), _p(kI.scales), max_blocks, _p(raw), n_raw, _p(raw_pos0), _p(q_pos),
        _p(sinks), _p(out), _p(idx_out), wp, wb, _s(stream)))


def csa_decode_noalloc(p: Params, batch: int, q, qI: Stored, w, kv: Stored, kI: Stored,
                       max_blocks: int, raw, n_raw: int, raw_pos0, q_pos, sinks, out, idx_out,
                       stream=None):
    """csa_decode without a workspace argument: the library's fixed device scratch
    is used instead.  Calls on one device must not overlap; requests larger than
    NOALLOC_SCRATCH_BYTES raise CsaError with status ERR_WORKSPACE."""
    _ok("csa_decode_noalloc", lib().csa_decode_noalloc(
        C.byref(p), batch, _p(q), _p(qI.data), _p(qI.scales), _p(w), _p(kv.data), _p(kv.scales),
        _p(kI.data), _p(kI.scales), max_blocks, _p(raw), n_raw, _p(raw_pos0), _p(q_pos),
        _p(sinks), _p(out), _p(idx_out), _s(stream)))


def csa_prefill(p: Params, batch: int, T: int, t0: int, raw, n_raw: int, raw_pos0: int, z, bias,
                q, qI: Stored, w, kv: Stored, kI: Stored, max_blocks: int, sinks, out, idx_out,
                workspace, stream=None):
    wp, wb = _ws(workspace)
    _ok("csa_prefill", lib().csa_prefill(
        C.byref(p), batch, T, t0, _p(raw), n_raw, raw_pos0, _p(z), _p(bias), _p(q), _p(qI.data),
        _p(qI.scales), _p(w), _p(kv.data), _p(kv.scales), _p(kI.data), _p(kI.scales),
        max_blocks, _p(sinks), _p(out), _p(idx_out), wp, wb, _s(stream)))


def csa_shard_select(p: Params, batch: int, qI: Stored, w, kI: Stored, n_entries: int, entry0: int, q_pos,
                     cand_scores, cand_ids, workspace, stream=None):
    wp, wb = _ws(workspace)
    _ok("csa_shard_select", lib().csa_shard_select(
        C.byref(p), batch, _p(qI.data), _p(qI.scales), _p(w), _p(kI.data), _p(kI.scales), n_entries, entry0,
        _p(q_pos), _p(cand_scores), _p(cand_ids), wp, wb, _s(stream)))


def csa_shard_attend(p: Params, batch: int, q, n_parts: int, cand_scores, cand_ids, kv: Stored,
                     n_entries: int, entry0: int, raw, n_raw: int, raw_pos0, q_pos, part_o, part_ml,
                     idx_out, workspace, stream=None):
    wp, wb = _ws(workspace)
    _ok("csa_shard_attend", lib().csa_shard_attend(
        C.byref(p), batch, _p(q), n_parts, _p(cand_scores), _p(cand_ids), _p(kv.data), _p(kv.scales),
        n_entries, entry0, _p(raw), n_raw, _p(raw_pos0), _p(q_pos), _p(part_o), _p(part_ml), _p(idx_out),
        wp, wb, _s(stream)))


def hca_shard_attend(p: Params, batch: int, q, kv: Stored, n_entries: int, entry0: int, raw, n_raw: int,
                     raw_pos0, q_pos, part_o, part_ml, workspace, stream=None):
    wp, wb = _ws(workspace)
    _ok("hca_shard_attend", lib().hca_shard_attend(
        C.byref(p), batch, _p(q), _p(kv.data), _p(kv.scales), n_entries, entry0, _p(raw), n_raw,
        _p(raw_pos0), _p(q_pos), _p(part_o), _p(part_ml), wp, wb, _s(stream)))


def attn_merge(p: Params, batch: int, n_parts: int, part_o, part_ml, sinks, out, stream=None):
    _ok("attn_merge", lib().attn_merge(C.byref(p), batch, n_parts, _p(part_o), _p(part_ml), _p(sinks),
                                       _p(out), _s(stream)))


def csa_device_status(reset: bool = True, stream=None) -> int:
    flags = C.c_uint32(0)
    _ok("csa_device_status", lib().csa_device_status(_s(stream), C.byref(flags), int(reset)))
    return flags.value


# ------------------------------------------------- grouped-head attention
def gqa_workspace_size(p: GqaParams, op: int, n_seq: int, n_tokens: int, n_ctx: int) -> int:
    return lib().csa_gqa_workspace_size(C.byref(p), op, n_seq, n_tokens, n_ctx)


def empty_paged(p: GqaParams, n_pages: int, device="cuda"):
    """Allocate (with torch) the key and value pages of a paged cache: (k, v), each
    [n_pages][n_kv_heads][page_size][head_dim] in p.cache_fmt."""
    lead = (n_pages, p.n_kv_heads, p.page_size)
    caches = []
    for _ in range(2):
        st = empty_stored(p.cache_fmt, n_pages * p.n_kv_heads * p.page_size, p.head_dim, device)
        st.data = st.data.view(*lead, -1)
        if st.scales is not None:
            st.scales = st.scales.view(*lead, -1)
        caches.append(st)
    return tuple(caches)


# These calls launch kernels of a few microseconds: their checks go by plain
# integers and by torch's own comparisons (a device object or a Stream costs a
# microsecond or more to make).
_dtypes = {}


def _dtype(fmt):
    """The torch type that elements of a format are passed in."""
    if not _dtypes:
        import torch
        _dtypes.update({F32: torch.float32, BF16: torch.bfloat16, FP8_S64: torch.uint8, "i32": torch.int32,
                        "i64": torch.int64, "f64": torch.float64})
    return _dtypes[fmt]


def _act_dtype(p):
    return _dtype(F32 if p.act_fmt == F32 else BF16)


def _rows_of(t, n, heads, p, name):
    """(pointer, token stride in elements) of [n][heads][d] rows; the rows of one token are
    dense, those of different tokens any stride apart."""
    d = p.head_dim
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.dtype != (act := _act_dtype(p)):
        raise ValueError(f"{name} must be {act}, got {t.dtype}")
    if t.shape != (n, heads, d):
        raise ValueError(f"{name} must be [{n}][{heads}][{d}], got {list(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != d):
        raise ValueError(f"the heads of one token of {name} must be dense")
    return t.data_ptr(), s[0] if n > 1 else heads * d


def _dense(t, shape, dtype, name):
    """Pointer of a dense tensor of this shape and type (None: no tensor)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    return _p(t)


def _check(dev, *specs):
    """Pointers of dense tensors of one device, each given as (tensor or None, shape, type, name)."""
    ptrs = []
    for spec in specs:
        t = spec[0]
        if t is None:
            ptrs.append(None)
        elif t.shape == spec[1] and t.dtype is spec[2] and t.get_device() == dev and t.is_contiguous():
            ptrs.append(t.data_ptr())
        else:
            _dense(*spec)
            raise ValueError(f"tensors on different devices: {spec[3]} on {t.device}, another on cuda:{dev}")
    return ptrs


def _cache_specs(p, hk, d, k_cache, v_cache, block_table, n_seq):
    """What _check is to see of a paged cache, in the calls' order, without the counts."""
    fmt = p.cache_fmt
    if k_cache.fmt != fmt or v_cache.fmt != fmt:
        raise ValueError(f"the caches are stored in formats {k_cache.fmt}, {v_cache.fmt}, the parameters name {fmt}")
    if block_table.dim() != 2 or block_table.shape[0] != n_seq:
        raise ValueError(f"block_table must be [{n_seq}][max_pages], got {list(block_table.shape)}")
    n_pages, page = k_cache.data.shape[0], p.page_size
    rows, dtype = (n_pages, hk, page, d), _dtype(fmt if fmt in (F32, BF16) else FP8_S64)
    ks = vs = scales = None
    if fmt == FP8_S64:
        ks, vs, scales = k_cache.scales, v_cache.scales, (n_pages, hk, page, d // 64)
        if ks is None or vs is None:
            raise ValueError("an FP8 cache needs its scales")
    f32, max_pages = _dtype(F32), block_table.shape[1]
    return ((k_cache.data, rows, dtype, "k_cache"), (ks, scales, f32, "k_cache scales"), (v_cache.data, rows, dtype, "v_cache"),
            (vs, scales, f32, "v_cache scales"), (block_table, (n_seq, max_pages), _dtype("i32"), "block_table"), n_pages,
            max_pages)


def _launch(fn, p, n, args, stream, dev):
    """Call an entry point with the tensors' device current (launches and the default stream go by
    the current device)."""
    import torch
    call = getattr(_lib or lib(), fn)
    if dev == torch.cuda.current_device():
        s = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)
        st = call(C.byref(p), n, *args, s)
    else:
        with torch.cuda.device(dev):
            st = call(C.byref(p), n, *args, _s(stream))
    if st:
        raise CsaError(fn, st)


def paged_append(p: GqaParams, n_seq: int, n_tokens: int, cu_q, pos0, q, k, v, inv_freq, q_out, k_out,
                 k_cache: Stored, v_cache: Stored, block_table, stream=None):
    """q [n_tokens][H][d] (or None), k, v [n_tokens][HK][d]; cu_q int32 [n_seq + 1] or None
    (one token per sequence); pos0 int64 [n_seq]; inv_freq float64 [rot_dim / 2] or None."""
    H, HK, d, act, rot = p.n_heads, p.n_kv_heads, p.head_dim, _act_dtype(p), p.rot_dim
    kp, kl = _rows_of(k, n_tokens, HK, p, "k")
    vp, vl = _rows_of(v, n_tokens, HK, p, "v")
    qp, ql = _rows_of(q, n_tokens, H, p, "q") if q is not None else (None, 0)
    dev = k.get_device()
    if v.get_device() != dev or (q is not None and q.get_device() != dev):
        raise ValueError("tensors on different devices: q, k, v")
    kc, ks, vc, vs, table, n_pages, max_pages = _cache_specs(p, HK, d, k_cache, v_cache, block_table, n_seq)
    cu, pos, f, qo, ko, kc, ks, vc, vs, table = _check(
        dev, (cu_q, (n_seq + 1,), _dtype("i32"), "cu_q"), (pos0, (n_seq,), _dtype("i64"), "pos0"),
        (inv_freq if rot > 0 else None, (rot // 2,), _dtype("f64"), "inv_freq"), (q_out, (n_tokens, H, d), act, "q_out"),
        (k_out, (n_tokens, HK, d), act, "k_out"), kc, ks, vc, vs, table)
    _launch("paged_append", p, n_seq, (n_tokens, cu, pos, qp, ql, kp, kl, vp, vl, f, qo, ko, kc, ks, vc, vs, n_pages, table,
                                       max_pages), stream, dev)


def paged_decode_attn(p: GqaParams, batch: int, q, k_cache: Stored, v_cache: Stored, block_table, q_pos, sinks,
                      out, workspace, stream=None):
    """q, out [batch][H][d]; q_pos int64 [batch]; sinks float32 [H] or None."""
    H, HK, d = p.n_heads, p.n_kv_heads, p.head_dim
    qp, ql = _rows_of(q, batch, H, p, "q")
    dev = q.get_device()
    kc, ks, vc, vs, table, n_pages, max_pages = _cache_specs(p, HK, d, k_cache, v_cache, block_table, batch)
    kc, ks, vc, vs, table, pos, snk, o, w = _check(
        dev, kc, ks, vc, vs, table, (q_pos, (batch,), _dtype("i64"), "q_pos"), (sinks, (H,), _dtype(F32), "sinks"),
        (out, (batch, H, d), q.dtype, "out"), _ws_spec(workspace))
    _launch("paged_decode_attn", p, batch, (qp, ql, kc, ks, vc, vs, n_pages, table, max_pages, pos, snk, o, w,
                                            _ws_bytes(workspace)), stream, dev)


def _ws_spec(ws):
    return (None,) if ws is None else (ws, ws.shape, ws.dtype, "workspace")


def _ws_bytes(ws):
    return 0 if ws is None else ws.nbytes


def prompt_attn(p: GqaParams, n_seq: int, q, k, v, cu_q, cu_k, sinks, out, workspace, stream=None):
    """q, out [n_q][H][d], k, v [n_k][HK][d]; cu_q, cu_k int32 [n_seq + 1]; sinks float32 [H]
    or None."""
    n_q, n_k, H, HK, i32 = q.shape[0], k.shape[0], p.n_heads, p.n_kv_heads, _dtype("i32")
    qp, ql = _rows_of(q, n_q, H, p, "q")
    kp, kl = _rows_of(k, n_k, HK, p, "k")
    vp, vl = _rows_of(v, n_k, HK, p, "v")
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("tensors on different devices: q, k, v")
    cq, ck, snk, o, w = _check(dev, (cu_q, (n_seq + 1,), i32, "cu_q"), (cu_k, (n_seq + 1,), i32, "cu_k"),
                               (sinks, (H,), _dtype(F32), "sinks"), (out, (n_q, H, p.head_dim), q.dtype, "out"),
                               _ws_spec(workspace))
    _launch("prompt_attn", p, n_seq, (qp, ql, n_q, kp, kl, vp, vl, n_k, cq, ck, snk, o, w, _ws_bytes(workspace)), stream, dev)
