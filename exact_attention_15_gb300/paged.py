"""torch layer of the paged key-value cache calls (``binding`` exports it).

Checks of arguments, allocation of the outputs and of the workspace, and the
C calls on torch's current stream; the computation runs in the library's CUDA
kernels. One call costs the host several microseconds, as much as the GPU needs
for a small one: ``csrc/paged_call.c`` makes the common calls (no given outputs,
the cache on the current device), and what it does not take, or everything where it
has not been built, goes through the checks here.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os

import torch

from .binding import _check, _check_tensor, library_path, load
from .build import CALLS_LIB

CACHE_BF16 = 0
CACHE_E4M3 = 1
_KINDS = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3}

_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
_bf16, _f64, _i32 = torch.bfloat16, torch.float64, torch.int32
_empty, _empty_like = torch.empty, torch.empty_like
_current_device = torch.cuda.current_device
# torch's current stream of a device as a pointer: a Stream object costs the host 3 us
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_calls = None


class _PythonCalls:
    """Stands in for the compiled calls where they have not been built: takes none."""

    @staticmethod
    def append(*args):
        return NotImplemented

    decode = forward = append


def _load_calls():
    """The compiled calls, bound to the library and torch (once), or their stand-in."""
    global _calls
    if _calls is None:
        path = os.path.join(os.path.dirname(library_path()), os.path.basename(CALLS_LIB))
        if not os.path.exists(path):
            _calls = _PythonCalls
            return _calls
        spec = importlib.util.spec_from_file_location(
            "_paged_call", path, loader=importlib.machinery.ExtensionFileLoader("_paged_call", path))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        lib = load()
        module.setup(*(ctypes.cast(getattr(lib, name), _P).value for name in (
            "attn_paged_append", "attn_paged_decode", "attn_paged_fwd", "attn_paged_call_workspace_bytes")), torch)
        _calls = module
    return _calls


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
        for name, t in (("k", k), ("v", v)):
            if t.dim() != 4 or t.dtype not in _KINDS or not t.is_cuda:
                raise ValueError(f"{name} must be a [num_pages, H_kv, page_size, d] bf16 or "
                                 f"float8_e4m3fn CUDA tensor, got {t.dtype} {tuple(t.shape)}")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must agree in shape, dtype and device")
        num_pages, H_kv, page_size, d = k.shape
        for name, t in (("k", k), ("v", v)):
            if num_pages > 0 and not t[0].is_contiguous():
                raise ValueError(f"{name} must be contiguous within a page")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is None:
                continue
            if k.dtype == _bf16:
                raise ValueError(f"{name}: a bf16 cache has no scales")
            _check_tensor(name, t, (H_kv,), torch.float32, k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.H_kv, self.page_size, self.d = num_pages, H_kv, page_size, d
        self.device = k.device
        self._index = k.get_device()
        self._kind = _KINDS[k.dtype]
        page = H_kv * page_size * d
        self._struct = _PagedCacheStruct(
            k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
            k.stride(0) if num_pages > 1 else page, v.stride(0) if num_pages > 1 else page,
            num_pages, page_size, H_kv, d, self._kind)
        self._ref = ctypes.addressof(self._struct)
        self._lib = load()
        self._calls = _load_calls()
        self._decode_bytes = self._lib.attn_paged_decode_workspace_bytes(d)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_seqs(cache, page_table, kv_lens, cu_seqlens, tokens):
    """Checks the arrays that describe the sequences. Returns their number and the
    page table's pointer, columns and row stride (one row may have any)."""
    index = cache._index
    if (kv_lens.dtype is not _i32 or kv_lens.dim() != 1 or not kv_lens.is_contiguous()
            or kv_lens.get_device() != index):
        raise ValueError(f"kv_lens must be a contiguous 1-D int32 tensor on {cache.device}")
    B = kv_lens.numel()
    if page_table.dtype is not _i32 or page_table.dim() != 2 or page_table.get_device() != index:
        raise ValueError(f"page_table must be a [{B}, max_pages] int32 tensor on {cache.device}")
    rows, cols = page_table.shape
    stride = cols
    if rows != B:
        raise ValueError(f"page_table has {rows} rows for {B} sequences")
    if not page_table.is_contiguous():
        stride = page_table.stride(0) if rows > 1 else cols
        if cols > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table must have contiguous rows")
    if cu_seqlens is None:
        if tokens != B:
            raise ValueError(f"without cu_seqlens there is one token per sequence: {tokens} for {B}")
    elif (cu_seqlens.dtype is not _i32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() != B + 1
          or not cu_seqlens.is_contiguous() or cu_seqlens.get_device() != index):
        raise ValueError(f"cu_seqlens must be a contiguous int32 tensor of {B + 1} entries on {cache.device}")
    return B, page_table.data_ptr(), cols, stride


def _tokens(name, t, cache):
    """Checks [tokens, heads, d] whose tokens are contiguous but may lie apart.
    Returns tokens, heads and the elements between tokens."""
    if t.dtype is _bf16 and t.get_device() == cache._index and t.dim() == 3:
        d = cache.d
        T, H, width = t.shape
        if width == d:
            if t.is_contiguous():
                return T, H, H * d
            a, b, c = t.stride()
            if c == 1 and (H <= 1 or b == d):
                return T, H, a if T > 1 else H * d
    raise ValueError(f"{name} must be a bf16 tensor [tokens, heads, {cache.d}] on {cache.device} whose tokens are "
                     f"contiguous, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _call(index, fn, *args):
    """fn(*args, stream) with torch's current stream of device `index`, which the C
    call takes as the current device."""
    if _current_device() == index:
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return fn(*args, _raw_stream(index))


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
    r = cache._calls.append(cache._ref, cache._index, q, k, v, page_table, kv_lens, cu_seqlens, inv_freq,
                            interleaved, q_out)
    if r is not NotImplemented:
        if type(r) is int:
            _check(r, "attn_paged_append")
        return r
    T, heads, ks = _tokens("k", k, cache)
    if heads != cache.H_kv:
        raise ValueError(f"k must be [tokens, {cache.H_kv} heads, d], got {heads} heads")
    Tv, heads, vs = _tokens("v", v, cache)
    if heads != cache.H_kv or Tv != T:
        raise ValueError(f"v must be like k, got {tuple(v.shape)} for {tuple(k.shape)}")
    B, table, cols, stride = _check_seqs(cache, page_table, kv_lens, cu_seqlens, T)
    rotary, freq = 0, None
    if inv_freq is not None:
        if (inv_freq.dtype is not _f64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()
                or inv_freq.get_device() != cache._index):
            raise ValueError(f"inv_freq must be a contiguous 1-D float64 tensor on {cache.device}")
        rotary, freq = 2 * inv_freq.numel(), inv_freq.data_ptr()
    H_q = qs = os = 0
    q_ptr = out_ptr = None
    if q is not None:
        Tq, H_q, qs = _tokens("q", q, cache)
        if Tq != T:
            raise ValueError(f"q must be of k's {T} tokens, got {Tq}")
        if q_out is None:
            q_out = _empty(q.shape, dtype=_bf16, device=cache.device) if rotary else q
            os = H_q * cache.d
        else:
            To, Ho, os = _tokens("q_out", q_out, cache)
            if To != T or Ho != H_q:
                raise ValueError(f"q_out must be like q, got {tuple(q_out.shape)} for {tuple(q.shape)}")
        if q_out is q and not rotary:
            H_q = 0  # nothing to write
        else:
            q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    status = _call(cache._index, cache._lib.attn_paged_append, cache._ref, q_ptr, k.data_ptr(), v.data_ptr(),
                   out_ptr, qs, ks, vs, os, T, B, H_q, None if cu_seqlens is None else cu_seqlens.data_ptr(), kv_lens.data_ptr(), table, cols,
                   stride, freq, rotary, bool(interleaved))
    if status:
        _check(status, "attn_paged_append")
    return q_out


def paged_workspace_bytes(cache, H_q, tokens=None, sequences=None) -> int:
    """Bytes of workspace of paged_forward for that many packed tokens and sequences,
    or of paged_decode without them."""
    if tokens is None:
        return cache._decode_bytes
    return load().attn_paged_fwd_workspace_bytes(tokens, sequences, H_q, cache.H_kv, cache.d, cache._kind)


def _outputs(cache, q, lse_shape, out, lse):
    H_q = q.shape[1]
    if H_q < 1 or H_q % cache.H_kv:
        raise ValueError(f"q has {H_q} heads, not a multiple of the cache's {cache.H_kv}")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if out is None:
        out = _empty_like(q)
    else:
        _check_tensor("out", out, q.shape, _bf16, cache.device)
    if lse is None:
        lse = _empty(lse_shape, device=cache.device, dtype=torch.float32)
    else:
        _check_tensor("lse", lse, lse_shape, torch.float32, cache.device)
    return out, lse


def _workspace(cache, workspace, size):
    if workspace is None:
        return _empty(size, dtype=torch.uint8, device=cache.device), size
    if not workspace.is_contiguous() or workspace.device != cache.device:
        raise ValueError("workspace must be a contiguous tensor on the cache's device")
    return workspace, workspace.numel() * workspace.element_size()


def paged_decode(cache, q, page_table, kv_lens, scale=None, out=None, lse=None, workspace=None):
    """Attention of one new token per sequence over the cache: q [B, H_q, d] bf16.
    Returns (o [B, H_q, d], lse [B, H_q]); a sequence without keys gives 0 and -inf.
    The default scale is 1/sqrt(d). The workspace (paged_workspace_bytes) is
    allocated with torch unless given."""
    if out is None and lse is None and workspace is None:
        r = cache._calls.decode(cache._ref, cache._index, cache.device, q, page_table, kv_lens, scale)
        if r is not NotImplemented:
            if type(r) is int:
                _check(r, "attn_paged_decode")
            return r
    T, H_q, _ = _tokens("q", q, cache)
    B, table, cols, stride = _check_seqs(cache, page_table, kv_lens, None, T)
    o, lse = _outputs(cache, q, (B, H_q), out, lse)
    lib = cache._lib
    ws, size = _workspace(cache, workspace, cache._decode_bytes)
    status = _call(cache._index, lib.attn_paged_decode, cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(),
                   B, H_q, kv_lens.data_ptr(), table, cols, stride,
                   1.0 / math.sqrt(cache.d) if scale is None else scale, ws.data_ptr(), size)
    if status:
        _check(status, "attn_paged_decode")
    return o, lse


def paged_forward(cache, q, page_table, kv_lens, cu_seqlens, scale=None, causal=True, out=None, lse=None,
                  workspace=None):
    """Attention of a chunk of new tokens per sequence over the cache, which holds
    them already: q [T, H_q, d] bf16, packed by cu_seqlens. With causal, the last new
    token sees all keys of its sequence and each one before sees one key less.
    Returns (o [T, H_q, d], lse [H_q, T]); rows behind the last sequence are not
    written."""
    if out is None and lse is None and workspace is None:
        r = cache._calls.forward(cache._ref, cache._index, cache.device, q, page_table, kv_lens, cu_seqlens, scale,
                                 causal)
        if r is not NotImplemented:
            if type(r) is int:
                _check(r, "attn_paged_fwd")
            return r
    T, H_q, _ = _tokens("q", q, cache)
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required (paged_decode takes one token per sequence)")
    B, table, cols, stride = _check_seqs(cache, page_table, kv_lens, cu_seqlens, T)
    o, lse = _outputs(cache, q, (H_q, T), out, lse)
    lib = cache._lib
    ws, size = _workspace(cache, workspace, lib.attn_paged_fwd_workspace_bytes(T, B, H_q, cache.H_kv, cache.d, cache._kind))
    status = _call(cache._index, lib.attn_paged_fwd, cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), T,
                   B, H_q, cu_seqlens.data_ptr(), kv_lens.data_ptr(), table, cols, stride, bool(causal),
                   1.0 / math.sqrt(cache.d) if scale is None else scale, ws.data_ptr(), size)
    if status:
        _check(status, "attn_paged_fwd")
    return o, lse
