"""Host-side checks of the paged key-value cache calls (no GPU): the C ABI's
refusals before anything is launched, and the binding's argument checks."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding, build, paged  # noqa: E402

OK, NULL, ALIGN, HEADDIM, SHAPE, GQA, WORKSPACE = 0, 1, 2, 3, 4, 5, 7
A = 0x10000  # a fake, aligned address: no call here may touch memory or a device


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _cache(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, num_pages=4, page_size=16, H_kv=2, d=64, type=0)
    a.update(kw)
    page = a["H_kv"] * a["page_size"] * a["d"]
    a.setdefault("k_page_stride", page)
    a.setdefault("v_page_stride", page)
    return paged._PagedCacheStruct(**a)


def _call(lib, name, cache=None, **kw):
    c = _cache() if cache is None else cache
    a = dict(q=A, k=A, v=A, q_out=A, o=A, lse=A, qs=256, ks=128, vs=128, os=256, T=3, B=3, H_q=4, cu=None, lens=A,
             table=A, max_pages=5, stride=5, freq=A, rotary=64, inter=0, causal=1, scale=0.125, ws=A, size=1 << 30)
    a.update(kw)
    ref = ctypes.addressof(c) if c != "null" else None
    if name == "append":
        return lib.attn_paged_append(ref, a["q"], a["k"], a["v"], a["q_out"], a["qs"], a["ks"], a["vs"], a["os"], a["T"],
                                     a["B"], a["H_q"], a["cu"], a["lens"], a["table"], a["max_pages"], a["stride"],
                                     a["freq"], a["rotary"], a["inter"], None)
    if name == "decode":
        return lib.attn_paged_decode(ref, a["q"], a["o"], a["lse"], a["B"], a["H_q"], a["lens"], a["table"],
                                     a["max_pages"], a["stride"], a["scale"], a["ws"], a["size"], None)
    return lib.attn_paged_fwd(ref, a["q"], a["o"], a["lse"], a["T"], a["B"], a["H_q"], A if a["cu"] is None else a["cu"],
                              a["lens"], a["table"], a["max_pages"], a["stride"], a["causal"], a["scale"], a["ws"],
                              a["size"], None)


CACHES = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=A + 8), ALIGN), (dict(v=A + 8), ALIGN),
    (dict(type=1, k_scale=A + 2), ALIGN), (dict(d=32), HEADDIM), (dict(d=192), HEADDIM), (dict(type=2), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(H_kv=0, k_page_stride=1, v_page_stride=1), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=512), SHAPE), (dict(k_page_stride=2047), SHAPE),
    (dict(v_page_stride=2052), ALIGN), (dict(v_page_stride=1 << 39), SHAPE), (dict(type=1, k_page_stride=2056), ALIGN),
]


@pytest.mark.parametrize("name", ["append", "decode", "fwd"])
@pytest.mark.parametrize("case", range(len(CACHES)))
def test_cache_refusals(lib, name, case):
    kw, want = CACHES[case]
    assert _call(lib, name, _cache(**kw)) == want


@pytest.mark.parametrize("name", ["append", "decode", "fwd"])
def test_sequence_refusals(lib, name):
    assert _call(lib, name, "null") == NULL
    assert _call(lib, name, B=-1, T=-1) == SHAPE
    assert _call(lib, name, H_q=5) == GQA
    assert _call(lib, name, H_q=-2) == SHAPE
    assert _call(lib, name, max_pages=-1) == SHAPE
    assert _call(lib, name, stride=4) == SHAPE
    assert _call(lib, name, max_pages=1 << 27, stride=1 << 27) == SHAPE
    assert _call(lib, name, lens=None) == NULL
    assert _call(lib, name, table=None) == NULL
    assert _call(lib, name, lens=A + 2) == ALIGN
    assert _call(lib, name, table=A + 1) == ALIGN
    assert _call(lib, name, B=0, T=0) == OK  # nothing to do


def test_append_refusals(lib):
    assert _call(lib, "append", T=4) == SHAPE       # one token per sequence without offsets
    assert _call(lib, "append", B=0) == SHAPE
    for bad in (-16, 8, 72, 80):
        assert _call(lib, "append", rotary=bad) == SHAPE
    assert _call(lib, "append", freq=None) == NULL
    assert _call(lib, "append", freq=A + 4) == ALIGN
    for name in ("q", "k", "v", "q_out"):
        assert _call(lib, "append", **{name: None}) == NULL
        assert _call(lib, "append", **{name: A + 4}) == ALIGN
    for name, row in (("qs", 256), ("ks", 128), ("vs", 128), ("os", 256)):
        assert _call(lib, "append", **{name: row - 8}) == SHAPE
        assert _call(lib, "append", **{name: row + 4}) == ALIGN


@pytest.mark.parametrize("name", ["decode", "fwd"])
def test_attention_refusals(lib, name):
    assert _call(lib, name, H_q=0) == SHAPE
    assert _call(lib, name, scale=float("nan")) == SHAPE
    assert _call(lib, name, scale=float("inf")) == SHAPE
    for arg in ("q", "o", "lse"):
        assert _call(lib, name, **{arg: None}) == NULL
        assert _call(lib, name, **{arg: A + 8}) == ALIGN
    need = (lib.attn_paged_decode_workspace_bytes(64) if name == "decode" else
            lib.attn_paged_fwd_workspace_bytes(3, 3, 4, 2, 64, 0))
    assert need > 0
    c, wide = _cache(), dict(max_pages=10000, stride=10000)
    of_call = lambda pages: lib.attn_paged_call_workspace_bytes(ctypes.addressof(c), 3, 3, 4, name == "fwd", pages)  # noqa: E731
    assert of_call(10000) == need and of_call(5) == 0
    assert _call(lib, name, size=need - 1, **wide) == WORKSPACE
    assert _call(lib, name, ws=None, **wide) == WORKSPACE
    assert _call(lib, name, ws=A + 128, **wide) == ALIGN
    assert _call(lib, name, ws=A + 128) == ALIGN


def test_fwd_needs_offsets(lib):
    c = _cache()
    assert lib.attn_paged_fwd(ctypes.addressof(c), A, A, A, 3, 3, 4, None, A, A, 5, 5, 1, 0.1, A, 1 << 30, None) == NULL
    assert _call(lib, "fwd", cu=A + 2) == ALIGN


def test_workspace_bytes(lib):
    f = lib.attn_paged_fwd_workspace_bytes
    assert f(1, 1, 1, 1, 128, 0) > 0 and f(0, 0, 1, 1, 64, 1) > 0
    # fp16 queries for an e4m3 cache, where the call has many rows per sequence
    assert f(4096, 1, 8, 2, 128, 1) >= f(4096, 1, 8, 2, 128, 0) + 4096 * 8 * (2 * 128 + 4)
    for bad in ((-1, 1, 1, 1, 64, 0), (1, -1, 1, 1, 64, 0), (1, 1, 0, 1, 64, 0), (1, 1, 3, 2, 64, 0),
                (1, 1, 1, 0, 64, 0), (1, 1, 1, 1, 96, 0), (1, 1, 1 << 20, 1, 64, 0), (1, 1, 1, 1, 64, 2)):
        assert f(*bad) == 0
    c, of_call = _cache(), lib.attn_paged_call_workspace_bytes
    for bad in ((0, 0, 4, 0, 5), (3, 3, 0, 0, 5), (3, 3, 5, 0, 5), (3, 3, 4, 0, -1), (3, 2, 4, 0, 10000)):
        assert of_call(ctypes.addressof(c), *bad) == 0
    assert of_call(None, 3, 3, 4, 0, 10000) == 0
    assert lib.attn_paged_decode_workspace_bytes(64) > 0 and lib.attn_paged_decode_workspace_bytes(96) == 0


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


class _HostCache:
    """Stands in for a PagedCache so that the other arguments' checks run here."""
    device, d, H_kv, page_size, num_pages = torch.device("cpu"), 64, 2, 16, 4
    _index, _decode_bytes, _lib = -1, 256, None  # (host tensors report the index -1)
    _ref, _calls = 0, None  # set in the test below


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def test_cache_rejects_host_tensors_and_wrong_types():
    _raises("CUDA tensor", binding.PagedCache, _t(4, 2, 16, 64), _t(4, 2, 16, 64))
    _raises("CUDA tensor", binding.PagedCache, _t(4, 2, 16), _t(4, 2, 16))
    f = _t(4, 2, 16, 64, dtype=torch.float16)
    _raises("bf16 or", binding.PagedCache, f, f)


def test_binding_checks_sequences_and_tokens(lib):
    """Through both the compiled calls (which refuse to take any of these) and the
    checks behind them."""
    c, i32 = _HostCache(), torch.int32
    struct = _cache()
    c._ref, c._calls = ctypes.addressof(struct), paged._load_calls()
    q, k = _t(3, 4, 64), _t(3, 2, 64)
    lens, table, cu = _t(3, dtype=i32), _t(3, 5, dtype=i32), _t(4, dtype=i32)
    _raises("kv_lens", binding.paged_decode, c, q, table, lens.long())
    _raises("kv_lens", binding.paged_decode, c, q, table, _t(6, dtype=i32)[::2])
    _raises("page_table", binding.paged_decode, c, q, table[:2], lens)
    _raises("page_table", binding.paged_decode, c, q, table.long(), lens)
    _raises("contiguous rows", binding.paged_decode, c, q, _t(5, 3, dtype=i32).t(), lens)
    _raises("one token per sequence", binding.paged_decode, c, _t(4, 4, 64), table, lens)
    _raises("q must be", binding.paged_decode, c, _t(3, 4, 128), table, lens)
    _raises("q must be", binding.paged_decode, c, q.float(), table, lens)
    _raises("q must be contiguous", binding.paged_decode, c, _t(3, 8, 64)[:, :4], table, lens)
    _raises("not a multiple", binding.paged_decode, c, _t(3, 3, 64), table, lens)
    _raises("out must be", binding.paged_decode, c, q, table, lens, out=_t(3, 4, 32))
    _raises("lse must be", binding.paged_decode, c, q, table, lens, lse=_t(4, 3, dtype=torch.float32))
    _raises("workspace", binding.paged_decode, c, q, table, lens, workspace=_t(64, 64)[:, ::2])
    _raises("cu_seqlens is required", binding.paged_forward, c, q, table, lens, None)
    _raises("cu_seqlens must be", binding.paged_forward, c, q, table, lens, cu[:3])
    _raises("cu_seqlens must be", binding.paged_forward, c, q, table, lens, cu.long())
    _raises("lse must be", binding.paged_forward, c, q, table, lens, cu, lse=_t(3, 4, dtype=torch.float32))
    _raises("k must be", binding.paged_append, c, q, _t(3, 4, 64), k, table, lens)
    _raises("v must be", binding.paged_append, c, q, k, _t(2, 2, 64), table, lens)
    _raises("v must be", binding.paged_append, c, q, k, _t(3, 64, 2).transpose(1, 2), table, lens)
    _raises("q must be", binding.paged_append, c, _t(2, 4, 64), k, k, table, lens)
    _raises("inv_freq", binding.paged_append, c, q, k, k, table, lens, inv_freq=_t(32, dtype=torch.float32))
    _raises("q_out must be", binding.paged_append, c, q, k, k, table, lens, q_out=_t(3, 2, 64))
    _raises("q_out without q", binding.paged_append, c, None, k, k, table, lens, q_out=q)
