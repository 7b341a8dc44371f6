"""Block-sparse masked flash attention with the ring (out, lse) merge, for GB300.

A thin ctypes binding over ``libra_gb300.so`` (the C ABI of ``include/ra.h``).
Every function named ``ra_*`` here has the same name, arguments and meaning
as its C counterpart and only marshals arguments: torch tensors become device
pointers, ``stream=None`` becomes the current torch CUDA stream.  All work
runs in the library's CUDA kernels; there is no fallback: if the library has
not been built, every call raises.

The helpers at the bottom (``make_params``, ``build_mask``, ``forward``,
``backward``, ``permute``, ``unpermute``; for a paged cache ``new_kv_cache``,
``make_kv_cache``, ``kv_write``, ``kv_read``, ``make_paged_params``,
``paged_forward``) allocate outputs with torch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

__all__ = [
    "RA_OK", "RA_ERR_INVALID_ARG", "RA_ERR_UNSUPPORTED", "RA_ERR_CUDA", "RA_ERR_WORKSPACE",
    "RA_ERR_TIMEOUT", "RA_BF16", "RA_FP32", "RA_TILE", "RaError", "RaAttnParams", "RaBlockMask",
    "lib", "ra_last_error", "ra_version", "ra_set_wait_timeout_ns", "ra_block_mask_bytes",
    "ra_build_block_mask", "ra_attn_fwd_workspace_size", "ra_attn_fwd", "ra_merge_out_lse",
    "ra_attn_bwd_workspace_size", "ra_attn_bwd", "ra_attn_bwd_prep", "ra_attn_bwd_dkdv",
    "ra_attn_bwd_dq", "ra_attn_bwd_noalloc", "ra_attn_bwd_noalloc_max_workspace",
    "ra_permute_tokens", "ra_unpermute_tokens", "RA_STEP_SINKS", "RA_STEP_FIRST",
    "ra_attn_fwd_step", "ra_attn_bwd_step", "ra_cast_from_f32", "ra_add_f32",
    "ra_get_device_status", "ra_launch_count", "ra_selftest_wait_timeout", "make_params", "build_mask", "forward", "backward", "permute",
    "unpermute",
    "RA_E4M3", "RaKvCache", "RaPagedParams", "ra_kv_write", "ra_kv_read",
    "ra_attn_paged_workspace_size", "ra_attn_paged", "new_kv_cache", "make_kv_cache", "kv_write",
    "kv_read", "make_paged_params", "paged_forward",
]

RA_OK = 0
RA_ERR_INVALID_ARG = -1
RA_ERR_UNSUPPORTED = -2
RA_ERR_CUDA = -3
RA_ERR_WORKSPACE = -4
RA_ERR_TIMEOUT = -5
RA_BF16 = 0
RA_FP32 = 1
RA_E4M3 = 2
RA_TILE = 128
RA_STEP_SINKS = 1
RA_STEP_FIRST = 2

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libra_gb300.so")


class RaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class RaAttnParams(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Lq", ctypes.c_int), ("Lkv", ctypes.c_int),
        ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
        ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("soft_cap", ctypes.c_float),
        ("causal", ctypes.c_int), ("is_mqa", ctypes.c_int), ("n_virtual_shards", ctypes.c_int),
        ("pad_segment_id", ctypes.c_int),
        ("q_pos", ctypes.c_void_p), ("kv_pos", ctypes.c_void_p),
        ("q_seg", ctypes.c_void_p), ("kv_seg", ctypes.c_void_p),
        ("sinks", ctypes.c_void_p), ("local_mask", ctypes.c_void_p),
        ("block_q_dkv", ctypes.c_int),
    ]


class RaBlockMask(ctypes.Structure):
    _fields_ = [
        ("tile_class", ctypes.c_void_p), ("fwd_cnt", ctypes.c_void_p),
        ("fwd_idx", ctypes.c_void_p), ("bwd_cnt", ctypes.c_void_p),
        ("bwd_idx", ctypes.c_void_p), ("fwd_order", ctypes.c_void_p),
        ("bwd_order", ctypes.c_void_p), ("fwd_shard", ctypes.c_void_p),
        ("part_fwd", ctypes.c_void_p), ("part_bwd", ctypes.c_void_p),
        ("part_rows", ctypes.c_void_p), ("part_cols", ctypes.c_void_p),
        ("n_part", ctypes.c_void_p), ("dkv_class", ctypes.c_void_p), ("dkv_cnt", ctypes.c_void_p),
        ("dkv_idx", ctypes.c_void_p), ("dkv_slot", ctypes.c_void_p), ("dkv_order", ctypes.c_void_p),
        ("B", ctypes.c_int), ("nq", ctypes.c_int),
        ("nk", ctypes.c_int), ("n_shards", ctypes.c_int), ("part_cap", ctypes.c_int),
        ("key", ctypes.c_uint64),
    ]


class RaKvCache(ctypes.Structure):
    """A paged cache; made by ``make_kv_cache``, the tensors are its attributes
    ``k_pages``, ``v_pages``, ``k_exps``, ``v_exps`` (the last two None for bf16)."""
    _fields_ = [
        ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p), ("v_exp", ctypes.c_void_p),
    ]


class RaPagedParams(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("Lq", ctypes.c_int), ("Hq", ctypes.c_int), ("dtype", ctypes.c_int),
        ("scale", ctypes.c_float), ("soft_cap", ctypes.c_float), ("causal", ctypes.c_int),
        ("max_pages", ctypes.c_int), ("prefix_pages", ctypes.c_int),
        ("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("q_len", ctypes.c_void_p),
        ("prefix_table", ctypes.c_void_p), ("prefix_len", ctypes.c_void_p),
        ("sinks", ctypes.c_void_p),
    ]


_lock = threading.Lock()
_lib = None


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build the CUDA library first "
                    "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            P = ctypes.POINTER(RaAttnParams)
            M = ctypes.POINTER(RaBlockMask)
            vp, ci, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.ra_last_error.restype = ctypes.c_char_p
            L.ra_version.restype = ctypes.c_char_p
            L.ra_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
            L.ra_set_wait_timeout_ns.restype = None
            L.ra_block_mask_bytes.argtypes = [P]
            L.ra_block_mask_bytes.restype = sz
            L.ra_build_block_mask.argtypes = [P, vp, sz, M, vp]
            L.ra_attn_fwd_workspace_size.argtypes = [P]
            L.ra_attn_fwd_workspace_size.restype = sz
            L.ra_attn_fwd.argtypes = [P, vp, vp, vp, M, vp, vp, vp, sz, vp]
            L.ra_merge_out_lse.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, vp]
            L.ra_attn_bwd_workspace_size.argtypes = [P]
            L.ra_attn_bwd_workspace_size.restype = sz
            L.ra_attn_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, M, vp, vp, vp, vp, vp, sz, vp]
            L.ra_attn_bwd_prep.argtypes = [P, vp, vp, vp, vp, vp, sz, vp]
            L.ra_attn_bwd_dkdv.argtypes = [P, vp, vp, vp, vp, M, vp, vp, vp, sz, vp]
            L.ra_attn_bwd_dq.argtypes = [P, vp, vp, vp, vp, M, vp, vp, sz, vp]
            L.ra_permute_tokens.argtypes = [vp, vp, ci, ci, sz, ci, vp]
            L.ra_unpermute_tokens.argtypes = [vp, vp, ci, ci, sz, ci, vp]
            L.ra_attn_bwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, M, vp, vp, vp, vp, vp]
            L.ra_attn_fwd_step.argtypes = [P, vp, vp, vp, M, ci, vp, vp, vp, vp]
            L.ra_attn_bwd_step.argtypes = [P, vp, vp, vp, vp, M, vp, vp, vp, vp, sz, vp]
            L.ra_cast_from_f32.argtypes = [vp, vp, sz, ci, vp]
            L.ra_add_f32.argtypes = [vp, vp, sz, vp]
            L.ra_attn_bwd_noalloc_max_workspace.restype = sz
            L.ra_get_device_status.argtypes = [vp]
            L.ra_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp, vp]
            L.ra_launch_count.restype = ctypes.c_uint64
            KC = PP = vp  # RaKvCache, RaPagedParams: by reference or by address
            L.ra_kv_write.argtypes = [KC, vp, vp, ci, ci, ci, sz, sz, vp, ci, vp, vp, vp]
            L.ra_kv_read.argtypes = [KC, vp, ci, vp, ci, ci, vp, vp, ci, vp]
            L.ra_attn_paged_workspace_size.argtypes = [KC, PP]
            L.ra_attn_paged_workspace_size.restype = sz
            L.ra_attn_paged.argtypes = [KC, PP, vp, vp, vp, vp, sz, vp]
            _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != RA_OK:
        raise RaError(rc, ra_last_error())


# ------------------------------------------------------------- C entry points
def ra_last_error() -> str:
    return lib().ra_last_error().decode()


def ra_version() -> str:
    return lib().ra_version().decode()


def ra_set_wait_timeout_ns(ns: int) -> None:
    lib().ra_set_wait_timeout_ns(int(ns))


def ra_block_mask_bytes(params: RaAttnParams) -> int:
    n = lib().ra_block_mask_bytes(ctypes.byref(params))
    if n == 0:
        raise RaError(RA_ERR_INVALID_ARG, ra_last_error())
    return int(n)


def ra_build_block_mask(params, buf, mask: RaBlockMask | None = None, stream=None) -> RaBlockMask:
    m = mask if mask is not None else RaBlockMask()
    nbytes = buf.numel() * buf.element_size()
    _check(lib().ra_build_block_mask(ctypes.byref(params), _ptr(buf), nbytes, ctypes.byref(m),
                                     _stream(stream)))
    m._buf = buf  # keep the device buffer alive with the struct
    return m


def ra_attn_fwd_workspace_size(params) -> int:
    return int(lib().ra_attn_fwd_workspace_size(ctypes.byref(params)))


def ra_attn_fwd(params, q, k, v, mask, out, lse, ws=None, stream=None) -> None:
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ra_attn_fwd(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(mask),
                             _ptr(out), _ptr(lse), _ptr(ws), ws_bytes, _stream(stream)))


def ra_merge_out_lse(out, lse, block_out, block_lse, B, L, H, D, stream=None) -> None:
    _check(lib().ra_merge_out_lse(_ptr(out), _ptr(lse), _ptr(block_out), _ptr(block_lse),
                                  B, L, H, D, _stream(stream)))


def ra_attn_bwd_workspace_size(params) -> int:
    return int(lib().ra_attn_bwd_workspace_size(ctypes.byref(params)))


def ra_attn_bwd(params, q, k, v, out, lse, dout, mask, dq, dk, dv, dsinks, ws, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ra_attn_bwd(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                             _ptr(lse), _ptr(dout), ctypes.byref(mask), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(dsinks), _ptr(ws), ws_bytes, _stream(stream)))


def ra_attn_bwd_noalloc(params, q, k, v, out, lse, dout, mask, dq, dk, dv, dsinks, stream=None):
    """ra_attn_bwd with the library's built-in scratch instead of a workspace."""
    _check(lib().ra_attn_bwd_noalloc(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                     _ptr(lse), _ptr(dout), ctypes.byref(mask), _ptr(dq), _ptr(dk),
                                     _ptr(dv), _ptr(dsinks), _stream(stream)))


def ra_attn_bwd_noalloc_max_workspace() -> int:
    return int(lib().ra_attn_bwd_noalloc_max_workspace())


def _wsb(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def ra_attn_bwd_prep(params, out, lse, dout, dsinks, ws, stream=None):
    _check(lib().ra_attn_bwd_prep(ctypes.byref(params), _ptr(out), _ptr(lse), _ptr(dout),
                                  _ptr(dsinks), _ptr(ws), _wsb(ws), _stream(stream)))


def ra_attn_bwd_dkdv(params, q, k, v, dout, mask, dk, dv, ws, stream=None):
    _check(lib().ra_attn_bwd_dkdv(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                  ctypes.byref(mask), _ptr(dk), _ptr(dv), _ptr(ws), _wsb(ws),
                                  _stream(stream)))


def ra_attn_bwd_dq(params, q, k, v, dout, mask, dq, ws, stream=None):
    _check(lib().ra_attn_bwd_dq(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                ctypes.byref(mask), _ptr(dq), _ptr(ws), _wsb(ws), _stream(stream)))


def ra_attn_fwd_step(params, q, k, v, mask, flags, out_run, lse_run, out=None, stream=None):
    """One ring step of the forward: merge the chunk (k, v) into (out_run, lse_run)."""
    _check(lib().ra_attn_fwd_step(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v),
                                  ctypes.byref(mask), int(flags), _ptr(out_run), _ptr(lse_run),
                                  _ptr(out), _stream(stream)))


def ra_attn_bwd_step(params, q, k, v, dout, mask, dq_acc, dk_acc, dv_acc, ws, stream=None):
    """One ring step of the backward: += the pair's gradients into fp32 accumulators."""
    _check(lib().ra_attn_bwd_step(ctypes.byref(params), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                                  ctypes.byref(mask), _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc),
                                  _ptr(ws), _wsb(ws), _stream(stream)))


def ra_cast_from_f32(inp, out, n, dtype, stream=None) -> None:
    _check(lib().ra_cast_from_f32(_ptr(inp), _ptr(out), int(n), int(dtype), _stream(stream)))


def ra_add_f32(acc, x, n, stream=None) -> None:
    _check(lib().ra_add_f32(_ptr(acc), _ptr(x), int(n), _stream(stream)))


def ra_permute_tokens(inp, out, B, L, row_bytes, n_shards, stream=None) -> None:
    _check(lib().ra_permute_tokens(_ptr(inp), _ptr(out), B, L, row_bytes, n_shards,
                                   _stream(stream)))


def ra_unpermute_tokens(inp, out, B, L, row_bytes, n_shards, stream=None) -> None:
    _check(lib().ra_unpermute_tokens(_ptr(inp), _ptr(out), B, L, row_bytes, n_shards,
                                     _stream(stream)))


def ra_launch_count() -> int:
    return int(lib().ra_launch_count())


def ra_get_device_status(stream=None) -> int:
    return int(lib().ra_get_device_status(_stream(stream)))


def ra_selftest_wait_timeout(timeout_ns, gave_up, stream=None) -> None:
    """One in-kernel wait that can never complete gives up after timeout_ns;
    ``gave_up`` is a device int32 tensor of one element."""
    _check(lib().ra_selftest_wait_timeout(int(timeout_ns), _ptr(gave_up), _stream(stream)))


def ra_kv_write(cache, k, v, dtype, B, L, k_stride, v_stride, page_table, max_pages, start,
                count=None, stream=None) -> None:
    _check(lib().ra_kv_write(ctypes.byref(cache), _ptr(k), _ptr(v), dtype, B, L, k_stride,
                             v_stride, _ptr(page_table), max_pages, _ptr(start), _ptr(count),
                             _stream(stream)))


def ra_kv_read(cache, page_table, max_pages, kv_len, B, L, k, v, dtype, stream=None) -> None:
    _check(lib().ra_kv_read(ctypes.byref(cache), _ptr(page_table), max_pages, _ptr(kv_len), B, L,
                            _ptr(k), _ptr(v), dtype, _stream(stream)))


def ra_attn_paged_workspace_size(cache, params) -> int:
    n = lib().ra_attn_paged_workspace_size(ctypes.byref(cache), ctypes.byref(params))
    if n == 0:  # also refused by ra_attn_paged, with the code of the refusal
        raise RaError(RA_ERR_INVALID_ARG, ra_last_error())
    return int(n)


def ra_attn_paged(cache, params, q, out, lse, ws, stream=None) -> None:
    _check(lib().ra_attn_paged(ctypes.byref(cache), ctypes.byref(params), _ptr(q), _ptr(out),
                               _ptr(lse), _ptr(ws), _wsb(ws), _stream(stream)))


# ------------------------------------------------------------- helpers
_DT = {torch.bfloat16: RA_BF16, torch.float32: RA_FP32}


def make_params(q, k, *, scale, causal=False, soft_cap=0.0, n_virtual_shards=1, is_mqa=False,
                pad_segment_id=-1, q_pos=None, kv_pos=None, q_seg=None, kv_seg=None,
                sinks=None, local_mask=None, block_q_dkv=0) -> RaAttnParams:
    """Params for q (B,Lq,Hq,D) and k (B,Lkv,Hkv,D) tensors; keeps the
    position / segment / sink / local-mask tensors referenced by the struct
    alive.  ``local_mask``: (Lq/N, Lkv/N) uint8 device tensor (non-causal only).
    ``block_q_dkv``: 0 / 128, or 64 for the dK/dV stage's own 64-row grid."""
    B, Lq, Hq, D = q.shape
    Lkv, Hkv = k.shape[1], k.shape[2]
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    p = RaAttnParams(B, Lq, Lkv, Hq, Hkv, D, _DT[q.dtype], float(scale),
                     float(soft_cap or 0.0), int(bool(causal)), int(bool(is_mqa)),
                     int(n_virtual_shards), int(pad_segment_id), _ptr(q_pos), _ptr(kv_pos),
                     _ptr(q_seg), _ptr(kv_seg), _ptr(sinks), _ptr(local_mask), int(block_q_dkv))
    p._keep = (q_pos, kv_pos, q_seg, kv_seg, sinks, local_mask)
    return p


def build_mask(params, device=None, stream=None) -> RaBlockMask:
    n = ra_block_mask_bytes(params)
    buf = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    return ra_build_block_mask(params, buf, stream=stream)


def forward(params, q, k, v, mask, stream=None, workspace=True):
    """Forward; with ``workspace`` the optional fp32 workspace that lets the
    library run two query heads per CTA is allocated (when it applies)."""
    B, Lq, Hq, D = q.shape
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    n = ra_attn_fwd_workspace_size(params) if workspace else 0
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n else None
    ra_attn_fwd(params, q, k, v, mask, out, lse, ws=ws, stream=stream)
    return out, lse


def backward(params, q, k, v, out, lse, dout, mask, stream=None):
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dsinks = (torch.empty(q.shape[2], dtype=torch.float32, device=q.device)
              if params.sinks else None)
    ws = torch.empty(ra_attn_bwd_workspace_size(params), dtype=torch.uint8, device=q.device)
    ra_attn_bwd(params, q, k, v, out, lse, dout, mask, dq, dk, dv, dsinks, ws, stream=stream)
    return dq, dk, dv, dsinks


def _rows(x):
    B, L = x.shape[0], x.shape[1]
    return B, L, x[0, 0].numel() * x.element_size()


def permute(x, n_shards, stream=None):
    """Zigzag permutation of axis 1 of a contiguous (B, L, ...) tensor."""
    x = x.contiguous()
    out = torch.empty_like(x)
    B, L, rb = _rows(x)
    ra_permute_tokens(x, out, B, L, rb, n_shards, stream=stream)
    return out


def unpermute(x, n_shards, stream=None):
    x = x.contiguous()
    out = torch.empty_like(x)
    B, L, rb = _rows(x)
    ra_unpermute_tokens(x, out, B, L, rb, n_shards, stream=stream)
    return out


# ------------------------------------------------------------- paged cache
_CACHE_DT = {torch.bfloat16: RA_BF16, torch.float8_e4m3fn: RA_E4M3}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(x, shape, name, index):
    """int32 tensors that the kernels read: dense, on the cache's device."""
    if x.dtype is torch.int32 and x.shape == shape and x.get_device() == index and x.is_contiguous():
        return
    if x.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, not {x.dtype}")
    _need(x.shape == shape, f"{name} has shape {tuple(x.shape)}, not {shape}")
    raise ValueError(f"{name} must be contiguous and on the cache's device")


def _here(index):
    """Whether device `index` is the current one.  The helpers then call with the handle of its
    current stream, and no Stream object around it: a small call's time is mostly Python's."""
    return index == torch._C._cuda_getDevice()


def _on(device, stream, run, *args):
    """run(*args, handle of the stream) on the tensors' device and on the caller's stream,
    allocations included, so that what is allocated is reused in that stream's order."""
    with torch.cuda.device(device):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        _need(stream is None or stream.device == device, "the stream is on another device than the cache")
        with torch.cuda.stream(stream):
            return run(*args, torch.cuda.current_stream().cuda_stream)


def make_kv_cache(k, v, k_exp=None, v_exp=None) -> RaKvCache:
    """A cache over existing tensors: k, v (n_pages, Hkv, page_size, D), bf16 or float8_e4m3fn,
    and for the latter k_exp, v_exp (n_pages, Hkv, page_size) uint8."""
    if k.dtype not in _CACHE_DT or v.dtype != k.dtype:
        raise TypeError(f"a cache is bfloat16 or float8_e4m3fn, not {k.dtype} and {v.dtype}")
    _need(k.dim() == 4 and k.shape == v.shape, "k and v must be (n_pages, Hkv, page_size, D)")
    quantised = k.dtype != torch.bfloat16
    _need((k_exp is not None) == quantised and (v_exp is not None) == quantised,
          "k_exp and v_exp belong to float8_e4m3fn caches")
    for x in (k, v, k_exp, v_exp):
        _need(x is None or (x.is_contiguous() and x.device == k.device),
              "cache tensors must be contiguous and on one device")
    for x in (k_exp, v_exp):
        if x is not None:
            if x.dtype != torch.uint8:
                raise TypeError(f"k_exp and v_exp must be uint8, not {x.dtype}")
            _need(x.shape == k.shape[:3], "k_exp and v_exp must be (n_pages, Hkv, page_size)")
    n, h, page, d = k.shape
    c = RaKvCache(n, page, h, d, _CACHE_DT[k.dtype], _ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp))
    c.k_pages, c.v_pages, c.k_exps, c.v_exps, c.device = k, v, k_exp, v_exp, k.device
    c._index = k.get_device()
    c._row = (h, d)
    c._sizes = (n, page, h, d, c.dtype, c._index)  # what params for it depend on
    c._ref = ctypes.addressof(c)
    return c


def new_kv_cache(n_pages, page_size, n_kv_heads, head_dim, dtype=torch.float8_e4m3fn,
                 device=None) -> RaKvCache:
    """An empty cache of ``n_pages`` pages (see ``make_kv_cache``)."""
    device = "cuda" if device is None else device
    shape = (n_pages, n_kv_heads, page_size, head_dim)
    if dtype not in _CACHE_DT:
        raise TypeError(f"a cache is bfloat16 or float8_e4m3fn, not {dtype}")
    k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype != torch.bfloat16 else dtype,
                        device=device).view(dtype) for _ in range(2))
    exps = [None, None] if dtype == torch.bfloat16 else [
        torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in range(2)]
    return make_kv_cache(k, v, *exps)


def _token_stride(shape, strides, name):
    B, L, H, D = shape
    sb, step, sh, sd = strides
    if L == 1:
        step = sb if B > 1 else H * D
    if not (sd == 1 and (sh == D or H == 1) and (B == 1 or sb == L * step) and step >= H * D):
        raise ValueError(
            f"{name}: a token's heads must be contiguous, and tokens and batches evenly spaced")
    return step


def kv_write(cache, k, v, page_table, start, count=None, stream=None) -> None:
    """Appends k, v (B, L, Hkv, D), bf16 or fp32, at positions start[b] + i of the sequences whose
    pages are in page_table (B, max_pages); of sequence b the first count[b] tokens (None: all).
    k and v may be slices along the head axis of a wider tensor.  No two tokens of a call may have
    the same place."""
    dt = _DT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise TypeError(f"k and v must both be bfloat16 or float32, not {k.dtype} and {v.dtype}")
    shape, index = k.shape, cache._index
    if not (len(shape) == 4 and v.shape == shape and shape[2:] == cache._row):
        raise ValueError(f"k and v must be (B, L, {cache.Hkv}, {cache.D}), of the same shape")
    if k.get_device() != index or v.get_device() != index:
        raise ValueError("k and v must be on the cache's device")
    strides = k.stride()
    ks = vs = _token_stride(shape, strides, "k")
    if v.stride() != strides:
        vs = _token_stride(shape, v.stride(), "v")
    B, L, _, _ = shape
    if B == 0 or L == 0:
        return
    pages = page_table.shape[-1]
    _ints(page_table, (B, pages), "page_table", index)
    _ints(start, (B,), "start", index)
    if count is not None:
        _ints(count, (B,), "count", index)
    args = (cache._ref, k.data_ptr(), v.data_ptr(), dt, B, L, ks, vs, page_table.data_ptr(), pages,
            start.data_ptr(), None if count is None else count.data_ptr())
    if stream is None and _here(index):
        rc = lib().ra_kv_write(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        rc = _on(cache.device, stream, lib().ra_kv_write, *args)
    if rc:
        _check(rc)


def _kv_read(cache, page_table, pages, kv_len, B, L, dtype, dt, s):
    k = torch.empty((B, L) + cache._row, dtype=dtype, device=cache.device)
    v = torch.empty_like(k)
    if B and L:
        _check(lib().ra_kv_read(cache._ref, page_table.data_ptr(), pages, kv_len.data_ptr(), B, L,
                                k.data_ptr(), v.data_ptr(), dt, s))
    return k, v


def kv_read(cache, page_table, kv_len, L, dtype=torch.bfloat16, stream=None):
    """k, v (B, L, Hkv, D) of the sequences' cached tokens; rows behind kv_len[b] are 0."""
    dt = _DT.get(dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {dtype}")
    index, (B, pages) = cache._index, page_table.shape
    _ints(page_table, (B, pages), "page_table", index)
    _ints(kv_len, (B,), "kv_len", index)
    args = cache, page_table, pages, kv_len, B, L, dtype, dt
    if stream is None and _here(index):
        return _kv_read(*args, torch._C._cuda_getCurrentRawStream(index))
    return _on(cache.device, stream, _kv_read, *args)


def make_paged_params(cache, q, page_table, kv_len, *, scale, causal=True, soft_cap=0.0, q_len=None,
                      sinks=None, prefix_table=None, prefix_len=None) -> RaPagedParams:
    """Params for queries like q (B, Lq, Hq, D) over ``cache``; they hold the tensors, which may be
    changed in place between calls (a page added, a length grown), and serve every layer whose
    cache has the same sizes and is on the same device.  prefix_len: an int32 tensor of one element."""
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    _need(q.dim() == 4 and q.shape[3] == cache.D, f"q must be (B, Lq, Hq, {cache.D})")
    B, Lq, Hq, _ = q.shape
    dev = cache.device
    _ints(page_table, (B, page_table.shape[-1]), "page_table", cache._index)
    _ints(kv_len, (B,), "kv_len", cache._index)
    if q_len is not None:
        _ints(q_len, (B,), "q_len", cache._index)
    _need((prefix_table is None) == (prefix_len is None),
          "prefix_table and prefix_len must come together")
    if prefix_table is not None:
        _ints(prefix_table, (prefix_table.shape[-1],), "prefix_table", cache._index)
        _ints(prefix_len, (1,), "prefix_len", cache._index)
    if sinks is not None:
        if sinks.dtype != torch.float32:
            raise TypeError(f"sinks must be float32, not {sinks.dtype}")
        _need(tuple(sinks.shape) == (Hq,) and sinks.is_contiguous() and sinks.device == dev,
              "sinks must be (Hq,), contiguous and on the cache's device")
    p = RaPagedParams(B, Lq, Hq, _DT[q.dtype], float(scale), float(soft_cap or 0.0),
                      int(bool(causal)), page_table.shape[1],
                      0 if prefix_table is None else prefix_table.shape[0], _ptr(page_table),
                      _ptr(kv_len), _ptr(q_len), _ptr(prefix_table), _ptr(prefix_len), _ptr(sinks))
    p._keep = (page_table, kv_len, q_len, prefix_table, prefix_len, sinks)
    p._like, p._lse = (q.shape, q.dtype), (B, Hq, Lq)
    p._ws = ra_attn_paged_workspace_size(cache, p) if B and Lq else 0
    p._cache = cache._sizes
    p._ref = ctypes.addressof(p)
    return p


def _paged_forward(params, q, cache, out, lse, ws, s):
    dev = cache.device
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(params._lse, dtype=torch.float32, device=dev)
    n = params._ws
    if n:
        if ws is None:
            # bare storage: a tensor around it would double the time of getting it
            w = torch.UntypedStorage(n, device=dev)
        else:
            w, n = ws, _wsb(ws)
        rc = lib().ra_attn_paged(cache._ref, params._ref, q.data_ptr(), out.data_ptr(),
                                 lse.data_ptr(), w.data_ptr(), n, s)
        if rc:
            _check(rc)
    return out, lse


def paged_forward(params, q, cache, out=None, lse=None, ws=None, stream=None):
    """Attention of q (B, Lq, Hq, D) over the cached tokens -> (out like q, lse (B, Hq, Lq) fp32).
    Given ``out`` / ``lse`` are written in place (rows behind q_len stay as they are); ``ws``: a
    workspace to use instead of a new one, uint8, of ra_attn_paged_workspace_size elements.
    For serving: no gradient is recorded."""
    index, like = cache._index, params._like
    if (q.shape, q.dtype) != like or not q.is_contiguous():
        raise ValueError("q must be contiguous, of the shape and dtype the params were made for")
    if cache._sizes != params._cache:
        raise ValueError("the params were made for a cache of other sizes, or on another device")
    if q.get_device() != index:
        raise ValueError("q must be on the cache's device")
    if out is not None and not ((out.shape, out.dtype) == like and out.get_device() == index
                                and out.is_contiguous()):
        raise ValueError("out must be like q")
    if lse is not None and not (lse.shape == params._lse and lse.dtype is torch.float32
                                and lse.get_device() == index and lse.is_contiguous()):
        raise ValueError("lse must be (B, Hq, Lq) fp32")
    if ws is not None and not (ws.get_device() == index and ws.is_contiguous()):
        raise ValueError("ws must be contiguous and on the cache's device")
    if stream is None and _here(index):
        return _paged_forward(params, q, cache, out, lse, ws,
                              torch._C._cuda_getCurrentRawStream(index))
    return _on(cache.device, stream, _paged_forward, params, q, cache, out, lse, ws)
