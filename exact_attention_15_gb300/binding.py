"""Thin Python binding over the C ABI in ``include/attn.h`` (ctypes).

The functions named like the C entry points take raw device pointers (ints)
and sizes exactly as the C functions do; ``forward`` / ``backward`` are
convenience wrappers that take torch CUDA tensors, allocate the outputs (and
the backward workspace) with torch, and pass pointers and torch's current
stream. Argument marshalling only: every step of the computation runs in the
library's CUDA kernels. There is no fallback: if the library has not been
built, or a call fails, an exception is raised.
"""

from __future__ import annotations

import ctypes
import math
import os

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libattn_gb300.so")
_lib = None

ATTN_STATUS = {
    0: "ATTN_OK", 1: "ATTN_ERR_NULL_PTR", 2: "ATTN_ERR_ALIGNMENT", 3: "ATTN_ERR_UNSUPPORTED_HEADDIM",
    4: "ATTN_ERR_BAD_SHAPE", 5: "ATTN_ERR_GQA_RATIO", 6: "ATTN_ERR_CAUSAL_SHAPE",
    7: "ATTN_ERR_WORKSPACE", 8: "ATTN_ERR_CUDA", 9: "ATTN_ERR_TIMEOUT", 10: "ATTN_ERR_NO_DEVICE",
    11: "ATTN_ERR_UNSUPPORTED_DEVICE", 12: "ATTN_ERR_SEQLENS", 13: "ATTN_ERR_PAGES",
}

# name -> (restype, argtypes)
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float
_Z = ctypes.c_size_t
_SIGS = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, ctypes.c_float, _P]),
    "attn_fwd_dims": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, ctypes.c_float, _P]),
    "attn_bwd_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                      ctypes.c_float, _I, _P, ctypes.c_size_t, _P]),
    "attn_bwd_dims_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "attn_bwd_dims": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P,
                           ctypes.c_float, _I, _P, ctypes.c_size_t, _P]),
    "attn_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                              ctypes.c_float, _I, _P]),
    "attn_paged_append": (_I, [_P, _P, _P, _P, _P, _L, _L, _L, _L, _I, _I, _I, _P, _P, _P, _I, _L, _P,
                               _I, _I, _P]),
    "attn_paged_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "attn_paged_decode": (_I, [_P, _P, _P, _P, _I, _I, _P, _P, _I, _L, _F, _P, _Z, _P]),
    "attn_paged_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _I, _L, _I, _F, _P, _Z, _P]),
    "attn_check": (_I, [_P]),
    "attn_status_string": (ctypes.c_char_p, [_I]),
    "attn_debug_exp2": (_I, [_P, _P, _I, _I, _P]),
    "attn_set_wait_limit": (ctypes.c_longlong, [ctypes.c_longlong]),
    "attn_set_bwd_variant": (_I, [_I]),
    "attn_set_fwd_variant": (_I, [_I]),
    "attn_debug_inject": (_I, [_I]),
    "attn_debug_stall": (_I, [_P]),
    "attn_debug_rescale_stats": (_I, [_P, _I]),
    "attn_debug_fwd_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, ctypes.c_longlong]),
    "attn_profile_enable": (_I, [_I]),
    "attn_profile_read": (_I, [_P, _I]),
}

KERNEL_NAMES = {1: "attn_fwd_kernel", 2: "attn_bwd_pre_kernel", 3: "attn_bwd_main_kernel",
                4: "attn_bwd_post_kernel", 5: "exp2_probe_kernel", 6: "stall_probe_kernel",
                7: "fwd_plan_kernel", 8: "attn_fwd_pair_kernel", 9: "attn_bwd_main_kernel_pass2",
                10: "bwd_plan_kernel", 11: "paged_append_kernel", 12: "paged_stream_kernel",
                13: "paged_join_kernel", 14: "paged_fwd_kernel", 15: "paged_plan_kernel"}
FAULT_NONE = 0
FAULT_SKIP_DQ_RELEASE = 1
BWD_ONE_CTA = 0
BWD_CTA_PAIR = 1
FWD_ONE_CTA = 0
FWD_CTA_PAIR = 1


class ProfileRecord(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("ms", ctypes.c_float)]


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {ATTN_STATUS.get(status, status)} ({status_string(status)})")


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads the shared library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"CUDA library not built: {_LIB_PATH} is missing "
                "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols():
    return list(_SIGS)


# ------------------------------------------------------------------ raw C entry points

def attn_fwd(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d, causal, seqlens, scale, stream) -> int:
    return load().attn_fwd(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d, int(causal), seqlens,
                           float(scale), stream)


def attn_fwd_dims(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d_qk, d_v, causal, seqlens, scale,
                  stream) -> int:
    return load().attn_fwd_dims(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d_qk, d_v, int(causal),
                                seqlens, float(scale), stream)


def attn_bwd_workspace_bytes(B, H_q, H_kv, N_q, N_k, d, varlen, deterministic) -> int:
    return load().attn_bwd_workspace_bytes(B, H_q, H_kv, N_q, N_k, d, int(varlen), int(deterministic))


def attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d, causal, seqlens,
             scale, deterministic, workspace, workspace_bytes, stream) -> int:
    return load().attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d,
                           int(causal), seqlens, float(scale), int(deterministic), workspace,
                           workspace_bytes, stream)


def attn_bwd_dims_workspace_bytes(B, H_q, H_kv, N_q, N_k, d_qk, d_v, varlen, deterministic) -> int:
    return load().attn_bwd_dims_workspace_bytes(B, H_q, H_kv, N_q, N_k, d_qk, d_v, int(varlen),
                                                int(deterministic))


def attn_bwd_dims(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d_qk, d_v, causal,
                  seqlens, scale, deterministic, workspace, workspace_bytes, stream) -> int:
    return load().attn_bwd_dims(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d_qk,
                                d_v, int(causal), seqlens, float(scale), int(deterministic),
                                workspace, workspace_bytes, stream)


def attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d, causal,
                     seqlens, scale, deterministic, stream) -> int:
    """attn_bwd served from the library's own fixed scratch buffer (no workspace,
    no allocation); for callers that cannot allocate device memory."""
    return load().attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N_q, N_k, d,
                                   int(causal), seqlens, float(scale), int(deterministic), stream)


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024


def attn_check(stream=None) -> int:
    return load().attn_check(stream)


def status_string(status: int) -> str:
    return load().attn_status_string(int(status)).decode()


attn_status_string = status_string


def attn_debug_exp2(x, y, n, mode, stream) -> int:
    return load().attn_debug_exp2(x, y, n, mode, stream)


def attn_debug_inject(fault: int) -> int:
    return load().attn_debug_inject(int(fault))


def attn_debug_rescale_stats(reset=True):
    """The forward's rescale counters (a library built with ATTN_COUNT_RESCALE=1):
    dict(warp_steps, warp_rescales, rows_moved, row_steps), or None when the
    library has no counters."""
    out = (ctypes.c_ulonglong * 4)()
    n = load().attn_debug_rescale_stats(ctypes.cast(out, _P), int(bool(reset)))
    if n < 0:
        raise AttnError(-n, "attn_debug_rescale_stats")
    if n == 0:
        return None
    return dict(warp_steps=out[0], warp_rescales=out[1], rows_moved=out[2], row_steps=out[3])


def attn_debug_stall(stream=None) -> int:
    return load().attn_debug_stall(stream)


FWD_ONE_CTA_PER_TILE = 0
FWD_STRIDING = 1
FWD_BALANCED_LIST = 2
FWD_CLAIMED = 3


def attn_debug_fwd_plan(B, H_q, H_kv, N_q, N_k, d_qk, d_v, causal, varlen, n_sm, want_lists=True):
    """The forward's launch plan for a shape, computed on the host (no GPU):
    dict(mode, grid, tiles, sec_heads, n_mblocks, pair_heads) and, for the balanced-list mode,
    'start' (per-CTA offsets, grid + 1) and 'tiles_of' (the concatenated lists).
    Raises on an argument error."""
    info = (ctypes.c_longlong * 6)()
    lib = load()
    st = lib.attn_debug_fwd_plan(B, H_q, H_kv, N_q, N_k, d_qk, d_v, int(causal), int(varlen),
                                 n_sm, ctypes.cast(info, _P), None, 0)
    if st != 0:
        raise ValueError(ATTN_STATUS.get(st, st))
    out = dict(mode=info[0], grid=info[1], tiles=info[2], sec_heads=info[3], n_mblocks=info[4],
               pair_heads=info[5])
    if want_lists and out["mode"] == FWD_BALANCED_LIST:
        cap = out["grid"] + 1 + out["tiles"]
        buf = (ctypes.c_int * cap)()
        st = lib.attn_debug_fwd_plan(B, H_q, H_kv, N_q, N_k, d_qk, d_v, int(causal), int(varlen),
                                     n_sm, ctypes.cast(info, _P), ctypes.cast(buf, _P), cap)
        if st != 0:
            raise ValueError(ATTN_STATUS.get(st, st))
        g = out["grid"]
        out["start"] = list(buf[:g + 1])
        out["tiles_of"] = list(buf[g + 1:cap])
    return out


def attn_set_wait_limit(cycles: int) -> int:
    return load().attn_set_wait_limit(int(cycles))


def attn_set_bwd_variant(variant: int) -> int:
    """BWD_ONE_CTA (default) or BWD_CTA_PAIR for the d = 128 backward; returns
    the previous selection (-1 for an unknown value)."""
    return load().attn_set_bwd_variant(int(variant))


def attn_set_fwd_variant(variant: int) -> int:
    """FWD_ONE_CTA (default) or FWD_CTA_PAIR for the d_qk = d_v = 128 forward;
    returns the previous selection (-1 for an unknown value)."""
    return load().attn_set_fwd_variant(int(variant))


def attn_profile_enable(enable: bool) -> int:
    return load().attn_profile_enable(int(bool(enable)))


def attn_profile_read(max_records: int = 65536):
    """Returns [(kernel_name, ms), ...] for launches since the last read."""
    buf = (ProfileRecord * max_records)()
    n = load().attn_profile_read(ctypes.cast(buf, ctypes.c_void_p), max_records)
    if n < 0:
        raise AttnError(-n, "attn_profile_read")
    return [(KERNEL_NAMES.get(buf[i].kernel, str(buf[i].kernel)), float(buf[i].ms)) for i in range(n)]


# ------------------------------------------------------------------ torch convenience layer

def _shape(q, k, cu_seqlens):
    if cu_seqlens is not None:
        T, H_q, d = q.shape
        H_kv = k.shape[1]
        return len(cu_seqlens) - 1, H_q, H_kv, T, k.shape[0], d
    B, N_q, H_q, d = q.shape
    return B, H_q, k.shape[2], N_q, k.shape[1], d


def _check_inputs(q, k, v, cu_seqlens):
    """Shapes first (so that a mismatch is reported as such), then dtype, device
    and layout: the C ABI takes sizes from q and k only, so v must match them."""
    import torch
    nd = 3 if cu_seqlens is not None else 4
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != nd:
            raise ValueError(f"{name} must have {nd} dimensions "
                             f"({'[T, H, d] with cu_seqlens' if nd == 3 else '[B, N, H, d]'}), "
                             f"got {tuple(t.shape)}")
    if v.shape[:-1] != k.shape[:-1]:
        raise ValueError(f"v {tuple(v.shape)} and k {tuple(k.shape)} differ outside the head dimension")
    if k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q and k head dimensions differ: {q.shape[-1]} vs {k.shape[-1]}")
    if nd == 4 and k.shape[0] != q.shape[0]:
        raise ValueError(f"q and k batch sizes differ: {q.shape[0]} vs {k.shape[0]}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    if cu_seqlens is not None:
        if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2
                or not cu_seqlens.is_contiguous() or cu_seqlens.device != q.device):
            raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor of at least two "
                             "entries on q's device")


def _check_tensor(name, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _lse_shape(B, H_q, N_q, cu_seqlens):
    return (H_q, N_q) if cu_seqlens is not None else (B, H_q, N_q)


def _stream_ptr():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(status, what):
    if status != 0:
        raise AttnError(status, what)


def forward(q, k, v, scale=None, causal=False, cu_seqlens=None, out=None, lse=None):
    """q [B, N_q, H_q, d_qk] (or packed [T, H_q, d_qk] with cu_seqlens), k with
    d_qk and v with d_v columns, bf16 CUDA tensors. Returns (o [.., d_v], lse).
    The default scale is 1/sqrt(d_qk)."""
    import torch
    _check_inputs(q, k, v, cu_seqlens)
    B, H_q, H_kv, N_q, N_k, d = _shape(q, k, cu_seqlens)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o_shape = q.shape[:-1] + (v.shape[-1],)
    if out is not None:
        _check_tensor("out", out, o_shape, torch.bfloat16, q.device)
    o = out if out is not None else torch.empty(o_shape, dtype=q.dtype, device=q.device)
    if lse is not None:
        _check_tensor("lse", lse, _lse_shape(B, H_q, N_q, cu_seqlens), torch.float32, q.device)
    else:
        lse = torch.empty(_lse_shape(B, H_q, N_q, cu_seqlens), dtype=torch.float32, device=q.device)
    cu_ptr = cu_seqlens.data_ptr() if cu_seqlens is not None else None
    d_v = v.shape[-1]
    _check(attn_fwd_dims(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                         B, H_q, H_kv, N_q, N_k, d, d_v, causal, cu_ptr, scale, _stream_ptr()),
           "attn_fwd_dims")
    return o, lse


def backward(q, k, v, o, lse, dout, scale=None, causal=False, cu_seqlens=None,
             deterministic=False, workspace=None):
    """Returns (dq, dk, dv): dq like q, dk like k, dv like v (q and k have d_qk
    columns, v, o and dout d_v). The workspace is allocated with torch unless
    given. The default scale is 1/sqrt(d_qk)."""
    import torch
    _check_inputs(q, k, v, cu_seqlens)
    B, H_q, H_kv, N_q, N_k, d = _shape(q, k, cu_seqlens)
    d_v = v.shape[-1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o_shape = q.shape[:-1] + (d_v,)
    _check_tensor("o", o, o_shape, torch.bfloat16, q.device)
    _check_tensor("dout", dout, o_shape, torch.bfloat16, q.device)
    _check_tensor("lse", lse, _lse_shape(B, H_q, N_q, cu_seqlens), torch.float32, q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    nbytes = attn_bwd_dims_workspace_bytes(B, H_q, H_kv, N_q, N_k, d, d_v, cu_seqlens is not None,
                                           deterministic)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous() or workspace.device != q.device:
        raise ValueError("workspace must be a contiguous tensor on q's device")
    cu_ptr = cu_seqlens.data_ptr() if cu_seqlens is not None else None
    _check(attn_bwd_dims(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                         dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                         B, H_q, H_kv, N_q, N_k, d, d_v, causal, cu_ptr, scale, deterministic,
                         workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         _stream_ptr()),
           "attn_bwd_dims")
    return dq, dk, dv


# ------------------------------------------------------------------ paged key-value cache

CACHE_BF16 = 0
CACHE_E4M3 = 1


class _PagedCacheStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("k_page_stride", _L),
                ("v_page_stride", _L), ("num_pages", _I), ("page_size", _I), ("H_kv", _I), ("d", _I),
                ("type", _I)]


class PagedCache:
    """The pages that hold the keys and values of many sequences.

    k and v: [num_pages, H_kv, page_size, d], bf16 or float8_e4m3fn, on the GPU,
    contiguous within a page (pages may be further apart, as in the halves of one
    [num_pages, 2, ...] tensor). k_scale and v_scale (e4m3): fp32 [H_kv], the
    factor a head's stored values stand for; None for 1. Keeps the tensors; their
    contents may change between calls."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        kinds = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3}
        for name, t in (("k", k), ("v", v)):
            if t.dim() != 4 or t.dtype not in kinds or not t.is_cuda:
                raise ValueError(f"{name} must be a [num_pages, H_kv, page_size, d] bf16 or "
                                 f"float8_e4m3fn CUDA tensor, got {t.dtype} {tuple(t.shape)}")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must agree in shape, dtype and device")
        num_pages, H_kv, page_size, d = k.shape
        for name, t in (("k", k), ("v", v)):
            if num_pages > 0 and t[0].stride() != (page_size * d, d, 1):
                raise ValueError(f"{name} must be contiguous within a page")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None:
                continue
            if k.dtype == torch.bfloat16:
                raise ValueError(f"{name}: a bf16 cache has no scales")
            _check_tensor(name, t, (H_kv,), torch.float32, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.H_kv, self.page_size, self.d = num_pages, H_kv, page_size, d
        self.device = k.device
        page = H_kv * page_size * d
        self._struct = _PagedCacheStruct(
            k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
            k.stride(0) if num_pages > 1 else page, v.stride(0) if num_pages > 1 else page,
            num_pages, page_size, H_kv, d, kinds[k.dtype])
        self._ref = ctypes.addressof(self._struct)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_paged(cache, page_table, kv_lens, cu_seqlens, tokens):
    """The arrays that describe the sequences; returns the number of sequences."""
    import torch
    dev, i32 = cache.device, torch.int32
    if kv_lens.dtype != i32 or kv_lens.dim() != 1 or not kv_lens.is_contiguous() or kv_lens.device != dev:
        raise ValueError(f"kv_lens must be a contiguous 1-D int32 tensor on {dev}")
    B = kv_lens.shape[0]
    if (page_table.dtype != i32 or page_table.dim() != 2 or page_table.shape[0] != B
            or page_table.device != dev or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError(f"page_table must be a [{B}, max_pages] int32 tensor with contiguous rows on {dev}")
    if cu_seqlens is None:
        if tokens != B:
            raise ValueError(f"without cu_seqlens there is one token per sequence: {tokens} for {B}")
    elif (cu_seqlens.dtype != i32 or cu_seqlens.shape != (B + 1,) or not cu_seqlens.is_contiguous()
            or cu_seqlens.device != dev):
        raise ValueError(f"cu_seqlens must be a contiguous int32 tensor of {B + 1} entries on {dev}")
    return B


def _table_args(page_table):
    """Pointer, columns and row stride (a single row, or none, may have any)."""
    rows, cols = page_table.shape
    return page_table.data_ptr(), cols, page_table.stride(0) if rows > 1 else cols


def _check_tokens(name, t, heads, d, tokens, device):
    import torch
    if (t.dim() != 3 or t.dtype != torch.bfloat16 or t.device != device
            or t.shape != (tokens if tokens is not None else t.shape[0], heads if heads is not None else t.shape[1], d)
            or (t.numel() and ((t.shape[1] > 1 and t.stride(1) != d) or t.stride(2) != 1))):
        raise ValueError(f"{name} must be a bf16 tensor [tokens, heads, {d}] on {device} whose tokens are "
                         f"contiguous, got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def _token_stride(t):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _on_device(device, call, *args):
    """call(*args, stream) with torch's current stream of `device`, which the C
    call takes as the current device."""
    import torch
    if torch.cuda.current_device() == device.index:
        return call(*args, torch.cuda.current_stream().cuda_stream)
    with torch.cuda.device(device):
        return call(*args, torch.cuda.current_stream().cuda_stream)


def paged_append(cache, q, k, v, page_table, kv_lens, cu_seqlens=None, inv_freq=None, interleaved=False,
                 q_out=None):
    """Appends new tokens to the cache, with the rotary position embedding.

    k and v [T, H_kv, d] and q [T, H_q, d] (or None), bf16, tokens any distance
    apart (views of one fused projection). kv_lens [B] counts each sequence's keys
    with its new tokens; cu_seqlens [B + 1] packs them (None: one token each).
    inv_freq: float64 [rotary_dim / 2] on the GPU, radians per position, or None to
    append as is. Pairs are the halves of the first rotary_dim elements, or
    neighbours with interleaved. Returns the turned q (written to q_out if given,
    which may be q; q itself without inv_freq and q_out)."""
    import torch
    dev, d = cache.device, cache.d
    _check_tokens("k", k, cache.H_kv, d, None, dev)
    T = k.shape[0]
    _check_tokens("v", v, cache.H_kv, d, T, dev)
    B = _check_paged(cache, page_table, kv_lens, cu_seqlens, T)
    rotary = 0
    if inv_freq is not None:
        if (inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()
                or inv_freq.device != dev):
            raise ValueError(f"inv_freq must be a contiguous 1-D float64 tensor on {dev}")
        rotary = 2 * inv_freq.shape[0]
    heads = 0
    result = q_out
    if q is not None:
        _check_tokens("q", q, None, d, T, dev)
        if q_out is not None:
            _check_tokens("q_out", q_out, q.shape[1], d, T, dev)
        elif rotary:
            result = torch.empty(q.shape, dtype=q.dtype, device=dev)
        else:
            result = q
        # without a rotation there is nothing to write when q stays where it is
        heads = 0 if result is q and not rotary else q.shape[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(_on_device(dev, load().attn_paged_append, cache._ref, _ptr(q) if heads else None, k.data_ptr(),
                      v.data_ptr(), _ptr(result) if heads else None, _token_stride(q) if heads else 0,
                      _token_stride(k), _token_stride(v), _token_stride(result) if heads else 0, T, B,
                      heads, _ptr(cu_seqlens), kv_lens.data_ptr(), *_table_args(page_table),
                      _ptr(inv_freq), rotary, int(interleaved)),
           "attn_paged_append")
    return result


def paged_workspace_bytes(tokens, sequences, H_q, H_kv, d) -> int:
    return load().attn_paged_workspace_bytes(tokens, sequences, H_q, H_kv, d)


def _paged_outputs(cache, q, B, lse_shape, out, lse, workspace):
    import torch
    dev = cache.device
    T, H_q = q.shape[0], q.shape[1]
    if H_q < 1 or H_q % cache.H_kv:
        raise ValueError(f"q has {H_q} heads, not a multiple of the cache's {cache.H_kv}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check_tensor("out", out, q.shape, torch.bfloat16, dev)
    if lse is None:
        lse = torch.empty(lse_shape, dtype=torch.float32, device=dev)
    else:
        _check_tensor("lse", lse, lse_shape, torch.float32, dev)
    if workspace is None:
        workspace = torch.empty(paged_workspace_bytes(T, B, H_q, cache.H_kv, cache.d), dtype=torch.uint8,
                                device=dev)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return out, lse, workspace


def paged_decode(cache, q, page_table, kv_lens, scale=None, out=None, lse=None, workspace=None):
    """Attention of one new token per sequence over the cache: q [B, H_q, d] bf16.
    Returns (o [B, H_q, d], lse [B, H_q]); a sequence without keys gives 0 and -inf.
    The default scale is 1/sqrt(d). The workspace (paged_workspace_bytes) is
    allocated with torch unless given."""
    _check_tokens("q", q, None, cache.d, None, cache.device)
    B = _check_paged(cache, page_table, kv_lens, None, q.shape[0])
    o, lse, ws = _paged_outputs(cache, q, B, q.shape[:2], out, lse, workspace)
    _check(_on_device(cache.device, load().attn_paged_decode, cache._ref, q.data_ptr(), o.data_ptr(),
                      lse.data_ptr(), B, q.shape[1], kv_lens.data_ptr(), *_table_args(page_table),
                      1.0 / math.sqrt(cache.d) if scale is None else scale, ws.data_ptr(),
                      ws.numel() * ws.element_size()),
           "attn_paged_decode")
    return o, lse


def paged_forward(cache, q, page_table, kv_lens, cu_seqlens, scale=None, causal=True, out=None, lse=None,
                  workspace=None):
    """Attention of a chunk of new tokens per sequence over the cache, which holds
    them already: q [T, H_q, d] bf16, packed by cu_seqlens. With causal, the last new
    token sees all keys of its sequence and each one before sees one key less.
    Returns (o [T, H_q, d], lse [H_q, T]); rows behind the last sequence are not
    written."""
    _check_tokens("q", q, None, cache.d, None, cache.device)
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required (paged_decode takes one token per sequence)")
    T = q.shape[0]
    B = _check_paged(cache, page_table, kv_lens, cu_seqlens, T)
    o, lse, ws = _paged_outputs(cache, q, B, (q.shape[1], T), out, lse, workspace)
    _check(_on_device(cache.device, load().attn_paged_fwd, cache._ref, q.data_ptr(), o.data_ptr(),
                      lse.data_ptr(), T, B, q.shape[1], cu_seqlens.data_ptr(), kv_lens.data_ptr(),
                      *_table_args(page_table), int(causal),
                      1.0 / math.sqrt(cache.d) if scale is None else scale, ws.data_ptr(),
                      ws.numel() * ws.element_size()),
           "attn_paged_fwd")
    return o, lse
