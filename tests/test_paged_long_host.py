"""Host-side checks (no GPU) of pages with scales of their own, page bounds, selection and
lists of pages: the C ABI's refusals before anything is launched."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding, build, paged  # noqa: E402

OK, NULL, ALIGN, SHAPE, GQA, WORKSPACE = 0, 1, 2, 4, 5, 7
A = 0x10000  # a fake, aligned address: no call here may touch memory or a device


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _cache(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, num_pages=4, page_size=16, H_kv=2, d=64, type=3, k_exp=A, v_exp=A)
    a.update(kw)
    page = a["H_kv"] * a["page_size"] * a["d"]
    a.setdefault("k_page_stride", page)
    a.setdefault("v_page_stride", page)
    return paged._PagedCacheStruct(**a)


def _call(lib, name, cache=None, **kw):
    c = _cache() if cache is None else cache
    a = dict(q=A, bounds=A, pages=A, lens=A, o=A, lse=A, T=3, B=3, H_q=4, cu=None, kv=A, table=A, max_pages=5, stride=5,
             head=5, count=4, first=1, last=2, ws=A, size=1 << 30)
    a.update(kw)
    ref = ctypes.addressof(c) if c != "null" else None
    if name == "bounds":
        return lib.attn_paged_bounds(ref, a["bounds"], a["T"], a["B"], a["cu"], a["kv"], a["table"], a["max_pages"], a["stride"], None)
    if name == "select":
        return lib.attn_paged_select(ref, a["q"], a["bounds"], a["pages"], a["lens"], a["T"], a["B"], a["H_q"], a["cu"], a["kv"],
                                     a["table"], a["max_pages"], a["stride"], a["count"], a["first"], a["last"], None)
    return lib.attn_paged_decode_lists(ref, a["q"], a["o"], a["lse"], a["B"], a["H_q"], a["kv"], a["table"], a["max_pages"],
                                       a["stride"], a["head"], 0.125, a["ws"], a["size"], None)


@pytest.mark.parametrize("name", ["bounds", "select", "lists"])
def test_refusals(lib, name):
    assert _call(lib, name, "null") == NULL
    assert _call(lib, name, _cache(k_exp=None)) == NULL
    assert _call(lib, name, _cache(v_exp=None)) == NULL
    assert _call(lib, name, _cache(type=2)) == SHAPE
    assert _call(lib, name, _cache(page_size=24)) == SHAPE
    assert _call(lib, name, B=-1, T=-1) == SHAPE
    assert _call(lib, name, max_pages=-1) == SHAPE
    assert _call(lib, name, stride=4) == SHAPE
    assert _call(lib, name, kv=None) == NULL
    assert _call(lib, name, table=None) == NULL
    assert _call(lib, name, kv=A + 2) == ALIGN
    assert _call(lib, name, table=A + 1) == ALIGN
    assert _call(lib, name, B=0, T=0) == OK  # nothing to do


@pytest.mark.parametrize("name", ["bounds", "select"])
def test_packed_refusals(lib, name):
    assert _call(lib, name, T=4) == SHAPE  # one token per sequence without offsets
    assert _call(lib, name, B=0) == SHAPE
    assert _call(lib, name, cu=A + 2) == ALIGN
    assert _call(lib, name, bounds=None) == NULL
    assert _call(lib, name, bounds=A + 8) == ALIGN


def test_select_refusals(lib):
    assert _call(lib, "select", H_q=5) == GQA
    assert _call(lib, "select", H_q=0) == SHAPE
    assert _call(lib, "select", H_q=2 * 129) == GQA
    for bad in (dict(count=0, first=0, last=1), dict(first=-1), dict(last=0), dict(count=2), dict(first=1 << 30, last=1 << 30),
                dict(max_pages=65537, stride=65537), dict(count=1 << 27)):
        assert _call(lib, "select", **bad) == SHAPE, bad
    for arg in ("q", "pages", "lens"):
        assert _call(lib, "select", **{arg: None}) == NULL
    assert _call(lib, "select", q=A + 8) == ALIGN
    for arg in ("pages", "lens"):
        assert _call(lib, "select", **{arg: A + 2}) == ALIGN


def test_lists_refusals(lib):
    assert _call(lib, "lists", head=4) == SHAPE
    assert _call(lib, "lists", H_q=5) == GQA
    assert _call(lib, "lists", max_pages=10000, stride=10000, head=10000, size=100) == WORKSPACE


def test_sizes_of_workspaces(lib):
    for T, B in ((5, 5), (1000, 3)):
        assert lib.attn_paged_fwd_workspace_bytes(T, B, 8, 2, 128, 3) == lib.attn_paged_fwd_workspace_bytes(T, B, 8, 2, 128, 0)
    assert lib.attn_paged_fwd_workspace_bytes(5, 5, 8, 2, 128, 2) == 0


# ---------------------------------------------------------------- the binding's checks

class _Fake:
    """What the checks look at of a tensor that is on a GPU."""

    def __init__(self, t):
        self._t, self.is_cuda, self.device = t, True, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self._t, name)

    def __getitem__(self, i):
        return self._t[i]


def _new_cache(k_scale=None, v_scale=None, dtype=torch.float8_e4m3fn):
    k = _Fake(torch.zeros(4, 2, 16, 64).to(dtype))
    fake = lambda t: None if t is None else _Fake(t)  # noqa: E731
    return paged.PagedCache(k, k, k_scale=fake(k_scale), v_scale=fake(v_scale))


def test_scales_of_pages():
    e = lambda *s: torch.zeros(*s, dtype=torch.uint8).view(torch.float8_e8m0fnu)  # noqa: E731
    c = _new_cache(e(4, 2), e(4, 2))
    assert c._struct.type == 3 and c._struct.k_scale is None and c._struct.k_exp
    c = _new_cache(torch.ones(2), torch.ones(2))
    assert c._struct.type == 1 and c._struct.k_exp is None
    for bad in ((e(4, 2), None), (None, e(4, 2)), (e(4, 2), torch.ones(2)), (e(2), e(2)), (e(4, 3), e(4, 3)),
                (e(2, 4).t(), e(4, 2)), (torch.ones(4, 2), torch.ones(4, 2))):
        with pytest.raises(ValueError):
            _new_cache(*bad)
    with pytest.raises(ValueError):
        _new_cache(e(4, 2), e(4, 2), dtype=torch.bfloat16)


def test_argument_checks():
    c = _new_cache()
    i32 = lambda *s: _Fake(torch.zeros(*s, dtype=torch.int32))  # noqa: E731
    bf = lambda *s: _Fake(torch.zeros(*s, dtype=torch.bfloat16))  # noqa: E731
    good = dict(q=bf(3, 4, 64), bounds=bf(4, 2, 2, 64), page_table=i32(3, 5), kv_lens=i32(3), count=4, pages=i32(3, 2, 4))
    for bad in (dict(q=bf(3, 5, 64)), dict(q=bf(3, 4, 32)), dict(bounds=bf(4, 2, 64)), dict(bounds=bf(5, 2, 2, 64)),
                dict(bounds=_Fake(torch.zeros(4, 2, 2, 64))), dict(page_table=i32(2, 5)), dict(page_table=i32(3, 2, 5)),
                dict(kv_lens=i32(3, 1)), dict(count=0, keep_last=0), dict(keep_last=0), dict(keep_first=4), dict(q=bf(4, 4, 64)),
                dict(cu_seqlens=i32(3)), dict(pages=i32(3, 2, 5)), dict(pages=bf(3, 2, 4)), dict(lens=i32(4))):
        with pytest.raises(ValueError):
            paged.paged_select(c, **{**good, **bad})
    good = dict(bounds=bf(4, 2, 2, 64), page_table=i32(3, 5), kv_lens=i32(3))
    for bad in (dict(bounds=bf(4, 2, 2, 32)), dict(cu_seqlens=i32(4)), dict(tokens=4), dict(page_table=i32(3, 2, 5)),
                dict(cu_seqlens=i32(3), tokens=3)):
        with pytest.raises(ValueError):
            paged.paged_bounds(c, **{**good, **bad})
    good = dict(q=bf(3, 4, 64), page_table=i32(3, 2, 5), kv_lens=i32(3), out=bf(3, 4, 64))
    for bad in (dict(page_table=i32(3, 3, 5)), dict(page_table=i32(2, 2, 5)),
                dict(page_table=_Fake(torch.zeros(3, 5, 2, dtype=torch.int32).transpose(1, 2)))):
        with pytest.raises(ValueError):
            paged.paged_decode(c, **{**good, **bad})
