"""ctypes binding of libattn.so (include/attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  The low-level functions keep the C names (attn_fwd, attn_decode,
attn_combine, ...) and take integer device addresses; ``fwd``, ``decode`` and
``combine`` build the problem struct from torch tensors, allocate the outputs
and the workspace with torch, and call them on torch's current stream, or on
the cudaStream_t given as ``stream``: what a call allocates then belongs to that
stream, as under ``torch.cuda.stream``.
There is no CPU fallback: if the library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libattn.so")

ATTN_F32, ATTN_F16, ATTN_BF16 = 0, 1, 2
ATTN_MASKED_ROWS_NAN, ATTN_MASKED_ROWS_ZERO = 0, 1
ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED, ATTN_ERR_ALIGNMENT = 0, 1, 2, 3
ATTN_ERR_WORKSPACE, ATTN_ERR_CUDA, ATTN_ERR_DEVICE_TIMEOUT = 4, 5, 6
ATTN_OFFSET_DEFAULT = -(2**63)
ATTN_CAUSAL_FIXED, ATTN_CAUSAL_KLENS = 0, 1
ATTN_KLENS_COUNT, ATTN_KLENS_LAST_INDEX = 0, 1
ATTN_KV_AS_Q, ATTN_KV_INT8 = 0, 1
ATTN_KV_SCALE_TENSOR, ATTN_KV_SCALE_CHANNEL = 0, 1
ATTN_INJECT_NONE, ATTN_INJECT_DROP_FIRST_COPY = 0, 1
DTYPE_CODE = {"f32": ATTN_F32, "f16": ATTN_F16, "bf16": ATTN_BF16}
EXPORTS = ("attn_fwd_workspace_size", "attn_fwd", "attn_decode_workspace_size", "attn_decode", "attn_combine",
           "attn_device_status", "attn_status_string", "attn_version", "attn_decode_noalloc",
           "attn_decode_noalloc_max_scratch", "attn_decode_append", "attn_probe_ex2", "attn_test_inject",
           "attn_fwd_window", "attn_fwd_window_workspace_size", "attn_decode_paged",
           "attn_decode_paged_workspace_size", "attn_qkv_prep")


class attn_layout(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_int64), ("batch_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class attn_problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("k_len", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("causal_offset", ctypes.c_int64), ("masked_rows", ctypes.c_int32),
                ("q", attn_layout), ("k", attn_layout), ("v", attn_layout), ("o", attn_layout),
                ("mask", attn_layout), ("seg_batch_stride", ctypes.c_int64),
                ("lse_batch_stride", ctypes.c_int64), ("lse_head_stride", ctypes.c_int64),
                ("window_left", ctypes.c_int32), ("causal_align", ctypes.c_int32),
                ("k_lens_kind", ctypes.c_int32), ("softcap", ctypes.c_float),
                ("smooth_softmax", ctypes.c_int32), ("head_sink", ctypes.c_void_p),
                ("kv_dtype", ctypes.c_int32), ("kv_scale_kind", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("key_splits", ctypes.c_int32)]


class attn_pages(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64)]


class attn_prep(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seq_len", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("eps", ctypes.c_float), ("max_pos", ctypes.c_int32), ("cache_rows", ctypes.c_int32),
                ("q", attn_layout), ("k", attn_layout), ("v", attn_layout), ("q_out", attn_layout),
                ("k_out", attn_layout), ("v_out", attn_layout), ("pos_batch_stride", ctypes.c_int64),
                ("row_batch_stride", ctypes.c_int64), ("kv_dtype", ctypes.c_int32),
                ("kv_scale_kind", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} (status {code})")
        self.code = code


_lib = None


def lib():
    """Load libattn.so (raises when it has not been built: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m attention_attn_fwd_02_gb300.build`"
                               " (or __graft_entry__.build()); there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(attn_problem)
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
        L.attn_fwd_workspace_size.argtypes, L.attn_fwd_workspace_size.restype = [P], sz
        L.attn_decode_workspace_size.argtypes, L.attn_decode_workspace_size.restype = [P], sz
        L.attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_fwd.restype = ctypes.c_int
        L.attn_decode.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_decode.restype = ctypes.c_int
        L.attn_combine.argtypes = [i32, i32, i32, vp, vp, i32, vp, i64, vp, i32, vp]
        L.attn_combine.restype = ctypes.c_int
        L.attn_device_status.argtypes, L.attn_device_status.restype = [vp], ctypes.c_int
        L.attn_status_string.argtypes, L.attn_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        L.attn_version.argtypes, L.attn_version.restype = [], ctypes.c_int
        L.attn_decode_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.attn_decode_noalloc.restype = ctypes.c_int
        L.attn_decode_noalloc_max_scratch.argtypes, L.attn_decode_noalloc_max_scratch.restype = [], sz
        L.attn_decode_append.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_decode_append.restype = ctypes.c_int
        L.attn_probe_ex2.argtypes, L.attn_probe_ex2.restype = [i32, i32, vp, vp], ctypes.c_int
        L.attn_test_inject.argtypes, L.attn_test_inject.restype = [i32], ctypes.c_int
        PP, PG = ctypes.POINTER(attn_prep), ctypes.POINTER(attn_pages)
        L.attn_fwd_window_workspace_size.argtypes, L.attn_fwd_window_workspace_size.restype = [P, i32], sz
        L.attn_fwd_window.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_fwd_window.restype = ctypes.c_int
        L.attn_decode_paged_workspace_size.argtypes = [P, PG, i32]
        L.attn_decode_paged_workspace_size.restype = sz
        L.attn_decode_paged.argtypes = [P, PG, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_decode_paged.restype = ctypes.c_int
        L.attn_qkv_prep.argtypes = [PP, PG] + [vp] * 13
        L.attn_qkv_prep.restype = ctypes.c_int
        _lib = L
    return _lib


# ---- the C entry points, same names ---------------------------------------------


def attn_fwd_workspace_size(p: attn_problem) -> int:
    return lib().attn_fwd_workspace_size(ctypes.byref(p))


def attn_decode_workspace_size(p: attn_problem) -> int:
    return lib().attn_decode_workspace_size(ctypes.byref(p))


def attn_fwd(p, q, k, v, o, mask, seg, k_lens, lse, workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd(ctypes.byref(p), q, k, v, o, mask, seg, k_lens, lse, workspace, workspace_bytes, stream)


def attn_decode(p, q, k_cache, v_cache, o, mask, seg, k_lens, lse, workspace, workspace_bytes, stream) -> int:
    return lib().attn_decode(ctypes.byref(p), q, k_cache, v_cache, o, mask, seg, k_lens, lse, workspace,
                             workspace_bytes, stream)


def attn_decode_noalloc(p, q, k_cache, v_cache, o, mask, seg, k_lens, lse, stream) -> int:
    """attn_decode with the library's fixed device scratch array instead of a caller workspace,
    for callers that cannot allocate device memory (see include/attn.h)."""
    return lib().attn_decode_noalloc(ctypes.byref(p), q, k_cache, v_cache, o, mask, seg, k_lens, lse, stream)


def attn_decode_append(p, q, k_new, v_new, k_cache, v_cache, o, mask, k_lens, lse, workspace, workspace_bytes,
                       stream) -> int:
    return lib().attn_decode_append(ctypes.byref(p), q, k_new, v_new, k_cache, v_cache, o, mask, k_lens, lse,
                                    workspace, workspace_bytes, stream)


def attn_fwd_window_workspace_size(p: attn_problem, first_keys: int) -> int:
    return lib().attn_fwd_window_workspace_size(ctypes.byref(p), first_keys)


def attn_fwd_window(p, first_keys, q, k, v, o, mask, seg, k_lens, lse, workspace, workspace_bytes, stream) -> int:
    return lib().attn_fwd_window(ctypes.byref(p), first_keys, q, k, v, o, mask, seg, k_lens, lse, workspace,
                                 workspace_bytes, stream)


def attn_decode_paged_workspace_size(p: attn_problem, pages: attn_pages, first_keys: int) -> int:
    return lib().attn_decode_paged_workspace_size(ctypes.byref(p), pages, first_keys)


def attn_decode_paged(p, pages, first_keys, q, k_pool, v_pool, o, mask, k_lens, lse, workspace, workspace_bytes,
                      stream) -> int:
    return lib().attn_decode_paged(ctypes.byref(p), pages, first_keys, q, k_pool, v_pool, o, mask, k_lens, lse,
                                   workspace, workspace_bytes, stream)


def attn_qkv_prep(p, pages, q, k, v, q_weight, k_weight, cos, sin, positions, rows, q_out, k_out, v_out,
                  stream) -> int:
    return lib().attn_qkv_prep(ctypes.byref(p), pages, q, k, v, q_weight, k_weight, cos, sin, positions, rows, q_out,
                               k_out, v_out, stream)


def attn_probe_ex2(blocks, iters, sink, stream) -> int:
    """Launch the exponential-throughput micro-kernel (a measurement utility; see include/attn.h)."""
    return lib().attn_probe_ex2(blocks, iters, sink, stream)


def attn_test_inject(fault: int) -> int:
    """Arm the one-shot bounded-wait test fault (a test utility; see include/attn.h)."""
    return lib().attn_test_inject(fault)


def attn_decode_noalloc_max_scratch() -> int:
    return lib().attn_decode_noalloc_max_scratch()


def attn_combine(n_splits, rows, head_dim, part_o, part_lse, out_dtype, o, o_row_stride, lse, masked_rows,
                 stream) -> int:
    return lib().attn_combine(n_splits, rows, head_dim, part_o, part_lse, out_dtype, o, o_row_stride, lse,
                              masked_rows, stream)


def attn_device_status(stream=None) -> int:
    return lib().attn_device_status(stream)


def status_string(code: int) -> str:
    try:
        return lib().attn_status_string(code).decode()
    except RuntimeError:
        return f"status {code}"


def attn_version() -> int:
    return lib().attn_version()


# ---- problem construction ---------------------------------------------------------


def make_problem(d: dict) -> attn_problem:
    """attn_problem from a plain dict (the fields of the struct; layouts as 4-tuples)."""
    p = attn_problem()
    p.batch, p.heads, p.kv_heads = d["batch"], d["heads"], d["kv_heads"]
    p.q_len, p.k_len, p.head_dim = d["q_len"], d["k_len"], d["head_dim"]
    p.dtype = DTYPE_CODE[d["dtype"]] if isinstance(d["dtype"], str) else int(d["dtype"])
    p.scale = float(d.get("scale") or 0.0)
    p.causal = 1 if d.get("causal") else 0
    off = d.get("causal_offset")
    p.causal_offset = ATTN_OFFSET_DEFAULT if off is None else int(off)
    mr = d.get("masked_rows", "nan")
    p.masked_rows = ATTN_MASKED_ROWS_ZERO if mr in ("zero", ATTN_MASKED_ROWS_ZERO) else ATTN_MASKED_ROWS_NAN
    for name in ("q", "k", "v", "o"):
        setattr(p, name, attn_layout(*d[f"{name}_layout"]))
    p.mask = attn_layout(*(d.get("mask_layout") or (0, 0, 0, 0)))
    p.seg_batch_stride = int(d.get("seg_batch_stride", d["q_len"]))
    lb, lh = d.get("lse_layout") or (d["heads"] * d["q_len"], d["q_len"])
    p.lse_batch_stride, p.lse_head_stride = lb, lh
    w = d.get("window_left")
    p.window_left = -1 if w is None else int(w)
    p.causal_align = ATTN_CAUSAL_KLENS if d.get("causal_align") in ("klens", ATTN_CAUSAL_KLENS) else ATTN_CAUSAL_FIXED
    p.k_lens_kind = (ATTN_KLENS_LAST_INDEX if d.get("k_lens_kind") in ("last_index", ATTN_KLENS_LAST_INDEX)
                     else ATTN_KLENS_COUNT)
    p.softcap = float(d.get("softcap") or 0.0)
    p.smooth_softmax = 1 if d.get("smooth_softmax") else 0
    p.head_sink = d.get("head_sink_ptr")      # device address of float32 [heads], or None
    p.kv_dtype = ATTN_KV_INT8 if d.get("kv_dtype") in ("i8", ATTN_KV_INT8) else ATTN_KV_AS_Q
    p.kv_scale_kind = (ATTN_KV_SCALE_CHANNEL if d.get("kv_scale") in ("channel", ATTN_KV_SCALE_CHANNEL)
                       else ATTN_KV_SCALE_TENSOR)
    p.k_scale = d.get("k_scale_ptr")          # device addresses of float32 scales (int8 caches)
    p.v_scale = d.get("v_scale_ptr")
    p.key_splits = int(d.get("key_splits") or 0)   # attn_fwd key ranges: 0 = the library's plan
    return p


def make_pages(page_size: int, n_pages: int, table, table_stride: int) -> attn_pages:
    """attn_pages; table is the device address of the int32 page lists."""
    return attn_pages(page_size, n_pages, table, table_stride)


def make_prep(d: dict) -> attn_prep:
    """attn_prep from a plain dict (the fields of the struct; layouts as 4-tuples under
    '<field>_layout')."""
    p = attn_prep()
    for name in ("batch", "seq_len", "heads", "kv_heads", "head_dim", "rot_dim", "max_pos", "cache_rows"):
        setattr(p, name, int(d[name]))
    p.dtype = DTYPE_CODE[d["dtype"]] if isinstance(d["dtype"], str) else int(d["dtype"])
    p.interleaved, p.norm, p.eps = int(d.get("interleaved", 0)), int(d.get("norm", 1)), float(d.get("eps", 1e-6))
    for name in ("q", "k", "v", "q_out", "k_out", "v_out"):
        setattr(p, name, attn_layout(*d[f"{name}_layout"]))
    p.pos_batch_stride = int(d.get("pos_batch_stride", d["seq_len"]))
    p.row_batch_stride = int(d.get("row_batch_stride", d["seq_len"]))
    p.kv_dtype = ATTN_KV_INT8 if d.get("kv_dtype") in ("i8", ATTN_KV_INT8) else ATTN_KV_AS_Q
    p.kv_scale_kind = (ATTN_KV_SCALE_CHANNEL if d.get("kv_scale") in ("channel", ATTN_KV_SCALE_CHANNEL)
                       else ATTN_KV_SCALE_TENSOR)
    p.k_scale = d.get("k_scale_ptr")
    p.v_scale = d.get("v_scale_ptr")
    return p


def _ptr(t):
    return None if t is None else t.data_ptr()


def _torch():
    import torch
    return torch


def _dtype_name(t):
    torch = _torch()
    return {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[t.dtype]


def _layout4(t, heads_dim: int):
    """(offset, batch, head, row) strides of a 4-D tensor whose dims are [B, S, H, D] (heads_dim=2)
    or [B, H, S, D] (heads_dim=1); offset 0 relative to data_ptr()."""
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("expected a 4-D tensor with contiguous last dimension")
    if heads_dim == 2:
        return (0, t.stride(0), t.stride(2), t.stride(1))
    return (0, t.stride(0), t.stride(1), t.stride(2))


def _check(code, where):
    if code != ATTN_OK:
        raise AttnError(code, where)


def _empty(stream, device, shape, dtype):
    """torch.empty for a call that launches on `stream` (None: torch's current one).  The allocator hands a freed
    block on in the order of the stream it was allocated under, so that has to be the stream of the kernels."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    # (0 and 1 both name the legacy default stream)
    on = torch.cuda.default_stream(device) if stream in (0, 1) else torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(on):
        return torch.empty(shape, dtype=dtype, device=device)


def _check_same(q, *, ints=(), floats=(), **same):
    """Raise unless the tensors are on q's device, `same` have q's dtype, ints are int32 and floats float32."""
    torch = _torch()
    if not q.is_cuda:
        raise ValueError("expected CUDA tensors")
    for name, t in same.items():
        if t is not None and (t.dtype != q.dtype or t.device != q.device):
            raise ValueError(f"{name}: expected {q.dtype} on {q.device}, got {t.dtype} on {t.device}")
    for group, dt in ((ints, torch.int32), (floats, torch.float32)):
        for t in group:
            if t is not None and (t.dtype != dt or t.device != q.device):
                raise ValueError(f"expected {dt} on {q.device}, got {t.dtype} on {t.device}")


def _check_extents(B, H, Sq, keys, *, mask, lse, head_sink, k_lens):
    """Raise unless what the kernels index by (entry, head, row, key) covers the problem."""
    if mask is not None:
        if mask.dim() != 4 or (mask.shape[3] > 1 and mask.stride(3) != 1):
            raise ValueError("mask must be float32, 4-D, keys contiguous")
        if any(m not in (1, n) for m, n in zip(mask.shape, (B, H, Sq))) or mask.shape[3] < keys:
            raise ValueError(f"mask: expected [{B}|1, {H}|1, {Sq}|1, {keys} keys or more], got {tuple(mask.shape)}")
    if lse is not None and (lse.shape != (B, H, Sq) or (Sq > 1 and lse.stride(2) != 1)):
        raise ValueError(f"lse: expected [{B}, {H}, {Sq}], contiguous rows, got {tuple(lse.shape)}")
    if head_sink is not None and (head_sink.shape != (H,) or not head_sink.is_contiguous()):
        raise ValueError(f"head_sink: expected contiguous [{H}], got {tuple(head_sink.shape)}")
    if k_lens is not None and (k_lens.shape != (B,) or not k_lens.is_contiguous()):
        raise ValueError("k_lens: expected contiguous int32 [batch]")


def _check_scales(i8, G, D, k_scale, v_scale):
    """Raise unless int8 caches have two scales, or two for every kv head and channel."""
    if not i8:
        return
    if k_scale is None or v_scale is None:
        raise ValueError("int8 caches: expected k_scale and v_scale")
    if k_scale.numel() != v_scale.numel() or k_scale.numel() not in (1, G * D):
        raise ValueError(f"k_scale, v_scale: expected both of 1 or both of {G * D} elements, got {k_scale.numel()} and "
                         f"{v_scale.numel()}")
    if not (k_scale.is_contiguous() and v_scale.is_contiguous()):
        raise ValueError("k_scale, v_scale: expected contiguous tensors")


def _page_dims(pool, table, page_layout):
    """(kv heads, page size, layout) of a pool [pages, G, page_size, D] ('hnd') or [pages, page_size, G, D] ('nhd')."""
    if page_layout not in ("hnd", "nhd") or pool.dim() != 4:
        raise ValueError("expected a 4-D pool, page_layout 'hnd' or 'nhd'")
    if table.dim() != 2 or table.stride(1) != 1:
        raise ValueError("table: expected [batch, pages of an entry], contiguous rows")
    head, row = (1, 2) if page_layout == "hnd" else (2, 1)
    return pool.shape[head], pool.shape[row], _layout4(pool, head)


def fwd(q, k, v, *, layout="bshd", causal=False, causal_offset=None, scale=0.0, mask=None, seg=None,
        k_lens=None, masked_rows="nan", return_lse=False, out=None, lse=None, stream=None,
        window_left=None, causal_align="fixed", k_lens_kind="count", softcap=0.0, smooth_softmax=False,
        head_sink=None, key_splits=0, first_keys=0):
    """O (and LSE) for torch CUDA tensors.  layout 'bshd': Q [B,Sq,H,D], K/V [B,Sk,G,D];
    'bhsd': Q [B,H,Sq,D], K/V [B,G,Sk,D].  mask: float32 broadcastable 4-D [B|1, H|1, Sq|1, Sk]
    with contiguous keys; seg: int32 [B, Sq] or [Sq]; k_lens: int32 [B].  window_left: left
    window of causal local attention (None = off); causal_align: 'fixed' (one offset) or
    'klens' (each entry's diagonal right-aligned to its key length); k_lens_kind: 'count' or
    'last_index' (ONNX seqlens_k, count minus one).  softcap: cap of the scaled scores (0 = off);
    smooth_softmax / head_sink (float32 [H] CUDA tensor): the sink term of the denominator.
    key_splits: key ranges merged in range order (0 = the library's shape-only plan).
    first_keys: with window_left, the first keys of each row's span (of its segment, or of the
    cache) that stay visible behind the window (attn_fwd_window)."""
    torch = _torch()
    hd = 2 if layout == "bshd" else 1
    sd = 1 if layout == "bshd" else 2
    B, Sq, H, D = q.shape[0], q.shape[sd], q.shape[hd], q.shape[3]
    G, Sk = k.shape[hd], k.shape[sd]
    if out is None:
        out = _empty(stream, q.device, q.shape, q.dtype)
    d = dict(batch=B, heads=H, kv_heads=G, q_len=Sq, k_len=Sk, head_dim=D, dtype=_dtype_name(q), scale=scale,
             causal=causal, causal_offset=causal_offset, masked_rows=masked_rows,
             q_layout=_layout4(q, hd), k_layout=_layout4(k, hd), v_layout=_layout4(v, hd),
             o_layout=_layout4(out, hd), window_left=window_left, causal_align=causal_align,
             k_lens_kind=k_lens_kind, softcap=softcap, smooth_softmax=smooth_softmax,
             head_sink_ptr=_ptr(head_sink), key_splits=key_splits)
    if mask is not None:
        if mask.dtype != torch.float32 or mask.dim() != 4 or mask.stride(3) != 1:
            raise ValueError("mask must be float32, 4-D, keys contiguous")
        d["mask_layout"] = (0, mask.stride(0) if mask.shape[0] > 1 else 0,
                            mask.stride(1) if mask.shape[1] > 1 else 0, mask.stride(2) if mask.shape[2] > 1 else 0)
    if seg is not None:
        d["seg_batch_stride"] = 0 if seg.dim() == 1 else seg.stride(0)
    if return_lse and lse is None:
        lse = _empty(stream, q.device, (B, H, Sq), torch.float32)
    if lse is not None:
        d["lse_layout"] = (lse.stride(0), lse.stride(1))
    p = make_problem(d)
    if first_keys:
        _check_extents(B, H, Sq, Sk, mask=mask, lse=lse, head_sink=head_sink, k_lens=k_lens)
        if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D or out.shape != q.shape:
            raise ValueError("q, k, v and out disagree")
        if seg is not None and (seg.shape not in ((Sq,), (B, Sq)) or (Sq > 1 and seg.stride(-1) != 1)):
            raise ValueError("seg: expected [q_len] or [batch, q_len], contiguous rows")
        _check_same(q, k=k, v=v, out=out, ints=(seg, k_lens), floats=(mask, lse, head_sink))
        with torch.cuda.device(q.device):
            ws_bytes = attn_fwd_window_workspace_size(p, first_keys)
            if ws_bytes and mask is not None:
                ws_bytes += 4 * 16 * B * H * Sq + 256   # the sums of up to 16 parts
            ws = _empty(stream, q.device, ws_bytes, torch.uint8) if ws_bytes else None
            st = torch.cuda.current_stream(q.device).cuda_stream if stream is None else stream
            _check(attn_fwd_window(p, first_keys, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(mask), _ptr(seg),
                                   _ptr(k_lens), _ptr(lse), _ptr(ws), ws_bytes, st), "attn_fwd_window")
        return (out, lse) if return_lse else out
    ws_bytes = attn_fwd_workspace_size(p)
    ws = _empty(stream, q.device, ws_bytes, torch.uint8) if ws_bytes else None
    st = torch.cuda.current_stream(q.device).cuda_stream if stream is None else stream
    _check(attn_fwd(p, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(mask), _ptr(seg), _ptr(k_lens), _ptr(lse),
                    _ptr(ws), ws_bytes, st), "attn_fwd")
    return (out, lse) if return_lse else out


def decode(q, k_cache, v_cache, k_lens=None, *, scale=0.0, mask=None, masked_rows="nan", return_lse=False,
           out=None, lse=None, workspace=None, stream=None, window_left=None, k_lens_kind="count", softcap=0.0,
           smooth_softmax=False, head_sink=None, k_scale=None, v_scale=None):
    """Single-query decode: q [B, 1, H, D]; caches BNSH [B, G, cap, D]; k_lens int32 [B].
    window_left keeps only the last window_left + 1 valid keys (local attention);
    k_lens_kind 'last_index' takes ONNX seqlens_k (count minus one) as given.
    int8 caches take float32 k_scale / v_scale tensors of 1 (per cache) or
    G * D (per kv head and channel) elements."""
    torch = _torch()
    B, Sq, H, D = q.shape
    G, cap = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = _empty(stream, q.device, q.shape, q.dtype)
    d = dict(batch=B, heads=H, kv_heads=G, q_len=Sq, k_len=cap, head_dim=D, dtype=_dtype_name(q), scale=scale,
             causal=window_left is not None, causal_align="klens", window_left=window_left,
             k_lens_kind=k_lens_kind, softcap=softcap, smooth_softmax=smooth_softmax,
             head_sink_ptr=_ptr(head_sink), masked_rows=masked_rows, q_layout=_layout4(q, 2),
             kv_dtype="i8" if k_cache.dtype == torch.int8 else None,
             kv_scale="channel" if (k_scale is not None and k_scale.numel() > 1) else "tensor",
             k_scale_ptr=_ptr(k_scale), v_scale_ptr=_ptr(v_scale),
             k_layout=_layout4(k_cache, 1), v_layout=_layout4(v_cache, 1), o_layout=_layout4(out, 2))
    if mask is not None:
        d["mask_layout"] = (0, mask.stride(0) if mask.shape[0] > 1 else 0,
                            mask.stride(1) if mask.shape[1] > 1 else 0, mask.stride(2) if mask.shape[2] > 1 else 0)
    if return_lse and lse is None:
        lse = _empty(stream, q.device, (B, H, Sq), torch.float32)
    if lse is not None:
        d["lse_layout"] = (lse.stride(0), lse.stride(1))
    p = make_problem(d)
    ws_bytes = attn_decode_workspace_size(p)
    if workspace is None:
        workspace = _empty(stream, q.device, ws_bytes, torch.uint8)
    st = torch.cuda.current_stream(q.device).cuda_stream if stream is None else stream
    _check(attn_decode(p, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(mask), None, _ptr(k_lens),
                       _ptr(lse), _ptr(workspace), workspace.numel(), st), "attn_decode")
    return (out, lse) if return_lse else out


def decode_paged(q, k_pool, v_pool, table, k_lens=None, *, page_layout="hnd", scale=0.0, mask=None,
                 masked_rows="nan", return_lse=False, out=None, lse=None, workspace=None, stream=None,
                 window_left=None, first_keys=0, k_lens_kind="count", softcap=0.0, smooth_softmax=False,
                 head_sink=None, k_scale=None, v_scale=None, max_rows=None):
    """Single-query decode over a paged cache: q [B, 1, H, D]; pools [pages, G, page_size, D]
    ('hnd') or [pages, page_size, G, D] ('nhd'); table int32 [B, pages of an entry]: entry b's
    row r is row r % page_size of page table[b, r // page_size], and a value that names no page
    hides its rows.  max_rows: rows an entry can hold (default: what its list holds); a mask
    [B|1, H|1, 1, max_rows or more] covers them.  window_left
    and first_keys: keep the last window_left + 1 valid keys and the first first_keys ones.
    Everything else as for decode."""
    torch = _torch()
    B, Sq, H, D = q.shape
    G, ps, kl = _page_dims(k_pool, table, page_layout)
    _, _, vl = _page_dims(v_pool, table, page_layout)
    if v_pool.shape != k_pool.shape or k_pool.shape[3] != D or table.shape[0] != B:
        raise ValueError("q, pools and table disagree")
    rows = table.shape[1] * ps if max_rows is None else max_rows
    if rows > table.shape[1] * ps:
        raise ValueError("max_rows: the table holds fewer rows")
    if out is None:
        out = _empty(stream, q.device, q.shape, q.dtype)
    i8 = k_pool.dtype == torch.int8
    _check_extents(B, H, Sq, rows, mask=mask, lse=lse, head_sink=head_sink, k_lens=k_lens)
    _check_scales(i8, G, D, k_scale, v_scale)
    if out.shape != q.shape:
        raise ValueError("out: expected the queries' shape")
    kv = {} if i8 else dict(k_pool=k_pool, v_pool=v_pool)
    _check_same(q, out=out, ints=(table, k_lens), floats=(mask, lse, head_sink, k_scale, v_scale), **kv)
    if i8 and (v_pool.dtype != torch.int8 or k_pool.device != q.device or v_pool.device != q.device):
        raise ValueError("int8 pools: both int8, on the queries' device")
    d = dict(batch=B, heads=H, kv_heads=G, q_len=Sq, k_len=rows, head_dim=D, dtype=_dtype_name(q), scale=scale,
             causal=window_left is not None, causal_align="klens", window_left=window_left,
             k_lens_kind=k_lens_kind, softcap=softcap, smooth_softmax=smooth_softmax,
             head_sink_ptr=_ptr(head_sink), masked_rows=masked_rows, q_layout=_layout4(q, 2),
             kv_dtype="i8" if i8 else None,
             kv_scale="channel" if (k_scale is not None and k_scale.numel() > 1) else "tensor",
             k_scale_ptr=_ptr(k_scale), v_scale_ptr=_ptr(v_scale), k_layout=kl, v_layout=vl,
             o_layout=_layout4(out, 2))
    if mask is not None:
        d["mask_layout"] = (0, mask.stride(0) if mask.shape[0] > 1 else 0,
                            mask.stride(1) if mask.shape[1] > 1 else 0, 0)
    if return_lse and lse is None:
        lse = _empty(stream, q.device, (B, H, Sq), torch.float32)
    if lse is not None:
        d["lse_layout"] = (lse.stride(0), lse.stride(1))
    p, pages = make_problem(d), make_pages(ps, k_pool.shape[0], _ptr(table), table.stride(0))
    with torch.cuda.device(q.device):
        ws_bytes = attn_decode_paged_workspace_size(p, pages, first_keys)
        if workspace is None:
            workspace = _empty(stream, q.device, ws_bytes, torch.uint8)
        elif workspace.device != q.device or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous tensor on {q.device}")
        st = torch.cuda.current_stream(q.device).cuda_stream if stream is None else stream
        _check(attn_decode_paged(p, pages, first_keys, _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(out), _ptr(mask),
                                 _ptr(k_lens), _ptr(lse), _ptr(workspace), workspace.numel(), st),
               "attn_decode_paged")
    return (out, lse) if return_lse else out


def qkv_prep(q, k, v, k_cache, v_cache, table=None, *, page_layout="hnd", q_weight=None, k_weight=None, norm=True,
             eps=1e-6, cos=None, sin=None, interleaved=False, positions=None, rows=None, k_scale=None, v_scale=None,
             out=None, stream=None):
    """The step before attention: RMS norm of each head of Q and K, rotation of their first
    2 * cos.shape[1] elements (no rotation without cos and sin), and the write of K and V into
    the cache.  q [B, S, H, D], k and v [B, S, G, D] (slices of a packed projection are fine);
    caches [B, G, cap, D] without a table, pools as for decode_paged with one.  cos, sin float32
    [positions, rot / 2]; positions and rows int32 [B, S] (default: the token's index): where the
    angle is taken and which cache row K and V go to (out of range: not written).  int8 caches
    take float32 k_scale / v_scale as decode does.  Returns the prepared queries [B, S, H, D]."""
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4 or v.shape != k.shape or q.shape[:2] != k.shape[:2] or q.shape[3] != k.shape[3]:
        raise ValueError("expected q [B, S, H, D] and k, v [B, S, G, D]")
    B, S, H, D = q.shape
    G = k.shape[2]
    if out is None:
        out = _empty(stream, q.device, q.shape, q.dtype)
    i8 = k_cache.dtype == torch.int8
    kv = {} if i8 else dict(k_cache=k_cache, v_cache=v_cache)
    _check_scales(i8, G, D, k_scale, v_scale)
    _check_same(q, k=k, v=v, out=out, q_weight=q_weight, k_weight=k_weight, ints=(positions, rows, table),
                floats=(cos, sin, k_scale, v_scale), **kv)
    if i8 and (v_cache.dtype != torch.int8 or k_cache.device != q.device or v_cache.device != q.device):
        raise ValueError("int8 caches: both int8, on the queries' device")
    if table is None:
        if k_cache.dim() != 4 or k_cache.shape[:2] != (B, G):
            raise ValueError("expected caches [B, G, rows, D]")
        heads, cap, kl, vl, pages = G, k_cache.shape[2], _layout4(k_cache, 1), _layout4(v_cache, 1), None
    else:
        heads, ps, kl = _page_dims(k_cache, table, page_layout)
        _, _, vl = _page_dims(v_cache, table, page_layout)
        cap, pages = table.shape[1] * ps, make_pages(ps, k_cache.shape[0], _ptr(table), table.stride(0))
        if table.shape[0] != B:
            raise ValueError("table: expected one list per batch entry")
    if heads != G or k_cache.shape != v_cache.shape or k_cache.shape[3] != D or out.shape != q.shape:
        raise ValueError("caches or out disagree with q, k and v")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and (t.shape != (D,) or not t.is_contiguous()):
            raise ValueError(f"{name}: expected [head_dim]")
    if (cos is None) != (sin is None) or (cos is not None and (
            cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous())):
        raise ValueError("cos, sin: expected two contiguous float32 [positions, rot / 2]")
    for name, t in (("positions", positions), ("rows", rows)):
        if t is not None and (t.shape != (B, S) or (S > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name}: expected int32 [batch, tokens]")
    p = make_prep(dict(
        batch=B, seq_len=S, heads=H, kv_heads=G, head_dim=D, rot_dim=0 if cos is None else 2 * cos.shape[1],
        dtype=_dtype_name(q), interleaved=interleaved, norm=norm, eps=eps,
        max_pos=0 if cos is None else cos.shape[0], cache_rows=cap, q_layout=_layout4(q, 2), k_layout=_layout4(k, 2),
        v_layout=_layout4(v, 2), q_out_layout=_layout4(out, 2), k_out_layout=kl, v_out_layout=vl,
        pos_batch_stride=0 if positions is None else positions.stride(0),
        row_batch_stride=0 if rows is None else rows.stride(0), kv_dtype="i8" if i8 else None,
        kv_scale="channel" if (k_scale is not None and k_scale.numel() > 1) else "tensor",
        k_scale_ptr=_ptr(k_scale), v_scale_ptr=_ptr(v_scale)))
    with torch.cuda.device(q.device):
        st = torch.cuda.current_stream(q.device).cuda_stream if stream is None else stream
        _check(attn_qkv_prep(p, pages, _ptr(q), _ptr(k), _ptr(v), _ptr(q_weight), _ptr(k_weight), _ptr(cos),
                             _ptr(sin), _ptr(positions), _ptr(rows), _ptr(out), _ptr(k_cache), _ptr(v_cache), st),
               "attn_qkv_prep")
    return out


def combine(part_o, part_lse, *, out_dtype=None, masked_rows="nan", return_lse=False, stream=None):
    """Merge partials: part_o float32 [rows, n_splits, D], part_lse float32 [rows, n_splits]."""
    torch = _torch()
    rows, n, D = part_o.shape
    out_dtype = out_dtype or torch.float32
    out = _empty(stream, part_o.device, (rows, D), out_dtype)
    lse = _empty(stream, part_o.device, (rows,), torch.float32) if return_lse else None
    st = torch.cuda.current_stream(part_o.device).cuda_stream if stream is None else stream
    code = {torch.float32: ATTN_F32, torch.float16: ATTN_F16, torch.bfloat16: ATTN_BF16}[out_dtype]
    _check(attn_combine(n, rows, D, _ptr(part_o), _ptr(part_lse), code, _ptr(out), D, _ptr(lse),
                        ATTN_MASKED_ROWS_ZERO if masked_rows == "zero" else ATTN_MASKED_ROWS_NAN, st),
           "attn_combine")
    return (out, lse) if return_lse else out
