"""Page bounds, selection of pages by them, and attention over lists of pages of their
own for each KV head, against definitions in 64 bits."""

import math

import pytest
import torch

from paged_common import Cache, as_int, assert_attention, attention
from long_common import Pages, bounds_of, selected, values_of

pytestmark = pytest.mark.gpu


def _binding():
    from exact_attention_15_gb300 import binding
    return binding


def _ok():
    assert _binding().attn_check(None) == 0


def _cu(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


def _make(kind, lens, H_kv, d, page, **kw):
    return Pages(lens, H_kv, d, page, **kw) if kind == "pages" else Cache(lens, H_kv, d, page, kind=kind, **kw)


def _keys(c, kind, p):
    """Keys of page p, [H_kv, page, d] in 64 bits."""
    if kind == "pages":
        return values_of(c.k[p], c.k_exp[p])
    x = c.k[p].double()
    return x if kind == "bf16" else x * c.k_scale.double()[:, None, None]


# ---------------------------------------------------------------- bounds

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "pages"])
@pytest.mark.parametrize("new,ctx,H_kv,d,page", [
    ([1], [0], 1, 64, 16), ([1, 1, 1, 1], [15, 16, 0, 500], 3, 128, 16), ([40, 0, 1, 129], [3, 50, 0, 31], 2, 64, 32),
    ([300, 5], [0, 127], 2, 128, 128), ([700], [200], 1, 128, 256), ([64, 2], [64, 62], 5, 64, 64)])
def test_bounds(new, ctx, H_kv, d, page, kind):
    lens = [n + x for n, x in zip(new, ctx)]
    c = _make(kind, lens, H_kv, d, page, seed=sum(lens))
    bounds = torch.full((c.k.shape[0], H_kv, 2, d), 7.0, device="cuda", dtype=torch.bfloat16)
    want = bounds.clone()
    for b, n in enumerate(new):
        for i in range((lens[b] - n) // page, (lens[b] - 1) // page + 1) if n else []:
            p = c.ids[b][i]
            want[p] = bounds_of(_keys(c, kind, p), min(page, lens[b] - i * page)).float().to(torch.bfloat16)
    one = all(n == 1 for n in new)
    got = _binding().paged_bounds(c.handle(), bounds, c.table, c.kv_lens, cu_seqlens=None if one else _cu(new),
                                  tokens=None if one else sum(new) + 3)  # (rows behind the last sequence)
    _ok()
    assert got is bounds
    assert torch.equal(as_int(bounds + 0.0), as_int(want + 0.0))


def test_bounds_of_special_keys():
    """NaN makes its column's bounds NaN, infinities are bounds; a negative scale turns the order round."""
    c = Cache([20], 1, 64, 16, kind="bf16", seed=1)
    p = c.ids[0][0]
    c.k[p, 0, 3, 5], c.k[p, 0, 4, 6], c.k[p, 0, 5, 7] = math.nan, math.inf, -math.inf
    bounds = torch.zeros(c.k.shape[0], 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    _binding().paged_bounds(c.handle(), bounds, c.table, c.kv_lens, cu_seqlens=_cu([20]), tokens=20)
    x = c.k[p, 0]
    assert bool(bounds[p, 0, :, 5].isnan().all())
    rest = [i for i in range(64) if i != 5]
    assert torch.equal(bounds[p, 0, 0, rest], x.amin(0)[rest]) and torch.equal(bounds[p, 0, 1, rest], x.amax(0)[rest])
    c = Cache([20], 1, 64, 16, kind="e4m3", seed=1)
    c.k_scale.neg_()
    _binding().paged_bounds(c.handle(), bounds, c.table, c.kv_lens, cu_seqlens=_cu([20]), tokens=20)
    for i in range(2):
        p = c.ids[0][i]
        want = bounds_of(_keys(c, "e4m3", p), min(16, 20 - 16 * i))
        assert torch.equal(bounds[p], want.float().to(torch.bfloat16))
    _ok()


def test_bounds_bad_pages():
    c = Cache([20, 20], 1, 64, 16, seed=1)
    bounds = torch.full((c.k.shape[0], 1, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    c.table[0, 1] = c.k.shape[0]
    _binding().paged_bounds(c.handle(), bounds, c.table, c.kv_lens)
    assert _binding().attn_check(None) == 13
    untouched = [p for p in range(c.k.shape[0]) if p != c.ids[1][1]]
    assert bool((bounds[untouched] == 7).all())


# ---------------------------------------------------------------- selection

class Boxes:
    """Sequences whose pages have bounds, and keys that nothing reads."""

    def __init__(self, lens, H_kv, d, page, seed=0, width=None, make=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        used = [-(-n // page) for n in lens]
        n_pages = sum(used) + 2
        self.page, self.lens = page, lens
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        width = max([1] + used) if width is None else width
        table = torch.full((len(lens), width), -9, dtype=torch.int32)
        self.ids = []
        for b, n in enumerate(used):
            self.ids.append([order.pop() for _ in range(n)])
            table[b, :n] = torch.tensor(self.ids[b], dtype=torch.int32)
        self.table = table.cuda()
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        mid = torch.randn(n_pages, H_kv, d, generator=g, device="cuda")
        wide = torch.randn(n_pages, H_kv, 2, d, generator=g, device="cuda").abs()
        self.bounds = torch.stack((mid - wide[:, :, 0], mid + wide[:, :, 1]), 2).to(torch.bfloat16)
        if make:
            make(self)
        from exact_attention_15_gb300 import binding
        k = torch.empty(n_pages, H_kv, page, d, device="cuda", dtype=torch.bfloat16)
        self.handle = binding.PagedCache(k, k)


def _check(c, q, new, count, first=0, last=1, rows=None):
    """One call against the definition, token by token."""
    H_kv, d = c.bounds.shape[1], c.bounds.shape[3]
    T = q.shape[0]
    pages = torch.full((T, H_kv, count), -5, dtype=torch.int32, device="cuda")
    lens = torch.full((T,), -5, dtype=torch.int32, device="cuda")
    one = new is None
    new = [1] * len(c.lens) if one else new
    got = _binding().paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, count, cu_seqlens=None if one else _cu(new),
                                  keep_first=first, keep_last=last, pages=pages, lens=lens)
    assert got[0] is pages and got[1] is lens
    _ok()
    t = 0
    pages, lens = pages.cpu(), lens.tolist()
    for b, n in enumerate(new):
        for i in range(n):
            seen = c.lens[b] - n + i + 1
            want, keys = selected(q[t].view(H_kv, -1, d), c.bounds, c.ids[b], max(seen, 0), c.page, count, first, last)
            assert torch.equal(pages[t], want), (b, i, (pages[t] != want).nonzero()[:4].tolist())
            assert lens[t] == keys
            t += 1
    assert bool((pages[t:] == -5).all()) and lens[t:] == [-5] * (T - t)
    return pages


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("lens,H_kv,group,d,page,count,first,last", [
    ([1], 1, 1, 64, 16, 1, 0, 1), ([100], 1, 4, 128, 16, 3, 1, 1), ([0, 17, 4000, 333], 2, 4, 128, 16, 8, 0, 1),
    ([9000, 16, 5000], 4, 8, 64, 32, 20, 2, 3), ([70000], 2, 5, 128, 16, 64, 1, 2), ([3000] * 40, 8, 4, 128, 64, 16, 1, 1),
    ([2000], 1, 24, 64, 16, 30, 0, 1), ([2000, 1500], 1, 128, 128, 16, 17, 0, 2), ([5000], 3, 1, 64, 256, 7, 3, 3),
    ([6000, 100], 2, 2, 128, 32, 6, 2, 4), ([40000], 16, 1, 64, 64, 300, 1, 1)])
def test_select(lens, H_kv, group, d, page, count, first, last, seed):
    c = Boxes(lens, H_kv, d, page, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    q = torch.randn(len(lens), H_kv * group, d, generator=g, device="cuda", dtype=torch.bfloat16)
    _check(c, q, None, count, first, last)


@pytest.mark.parametrize("new,ctx", [([4, 4, 4], [0, 500, 3000]), ([1, 0, 7, 2], [900, 10, 0, 2000]), ([200], [1000])])
@pytest.mark.parametrize("H_kv,group,d,page,count", [(2, 4, 128, 16, 9), (1, 8, 64, 32, 4)])
def test_select_of_chunks(new, ctx, H_kv, group, d, page, count):
    """Each token of a chunk chooses among the pages that it sees; two rows behind the last sequence."""
    c = Boxes([n + x for n, x in zip(new, ctx)], H_kv, d, page, seed=3)
    q = torch.randn(sum(new) + 2, H_kv * group, d, device="cuda", dtype=torch.bfloat16)
    _check(c, q, new, count, 1, 1)


def test_select_padding_rows():
    """A sequence shorter than its rows: tokens at negative positions see nothing."""
    c = Boxes([3, 100], 1, 64, 16)
    q = torch.randn(12, 2, 64, device="cuda", dtype=torch.bfloat16)
    pages = _check(c, q, [6, 6], 4, 1, 1)
    assert bool((pages[:3] == -1).all())


@pytest.mark.parametrize("width", [65536, 9000, 300])
@pytest.mark.parametrize("tokens", [1, 70])
def test_select_behind_wide_tables(width, tokens):
    """Up to 65,536 pages a row, of which few or all are in use."""
    lens = [16 * width if width < 65536 or tokens == 1 else 16 * 30000] + [500] * (tokens - 1)
    c = Boxes(lens, 1, 64, 16, width=width)
    q = torch.randn(tokens, 4, 64, device="cuda", dtype=torch.bfloat16)
    _check(c, q, None, 40, 1, 1)


def _same(c):       # all pages alike: the lower ones
    c.bounds[:] = c.bounds[:1]


def _pairs(c):      # every page beside two equal ones
    c.bounds[:] = c.bounds[torch.arange(c.bounds.shape[0], device="cuda") // 3 * 3]


def _zeros(c):
    c.bounds.zero_()


def _far(c):        # one page far above the rest, the others close together
    c.bounds[:] = 1.0 + 0.01 * c.bounds.sign()
    c.bounds[c.ids[0][7]] *= 1e4


def _close(c):      # scores that differ in their last bits: bf16 values 2^-7 apart in one column
    n = c.bounds.shape[0]
    c.bounds[:] = c.bounds[:1]
    c.bounds[..., 0] = (1 + torch.arange(n, device="cuda") % 5 / 128).to(torch.bfloat16)[:, None, None]


def _tiny(c):       # products below the smallest 32-bit number
    c.bounds.mul_(2.0 ** -110)


def _huge(c):       # sums above the largest
    c.bounds.mul_(2.0 ** 126)


def _infinite(c):
    c.bounds[c.ids[0][9], :, 1] = math.inf
    c.bounds[c.ids[0][20], :, 0] = -math.inf


def _nan(c):        # above all
    c.bounds[c.ids[0][13], :, 0, 3] = math.nan
    c.bounds[c.ids[0][40]] = math.nan


@pytest.mark.parametrize("make", [_same, _pairs, _zeros, _far, _close, _tiny, _huge, _infinite, _nan])
@pytest.mark.parametrize("n,tokens", [(700, 1), (3000, 1), (700, 40)])
def test_select_of_special_bounds(make, n, tokens):
    c = Boxes([16 * n] + [3000] * (tokens - 1), 1, 64, 16, make=make)
    q = torch.randn(tokens, 3, 64, device="cuda", dtype=torch.bfloat16)
    if make is _infinite:  # (no product of zero and infinity, which is NaN)
        q = q.sign() * q.abs().clamp(min=0.1)
    if make is _tiny:
        q = q * 2.0 ** -50
    _check(c, q.to(torch.bfloat16), None, 30, 1, 1)


@pytest.mark.parametrize("make", [None, _same, _pairs, _zeros, _far, _close, _tiny, _huge, _infinite, _nan])
@pytest.mark.parametrize("d,group,count", [(64, 3, 9), (128, 4, 70), (128, 11, 5)])
def test_select_few_pages_for_many_tokens(make, d, group, count):
    """More than 1520 tokens and heads behind a table of up to 160 pages."""
    c = Boxes([1536, 1, 40, 700, 0, 1300, 1535, 160] * 26, 8, d, 16, make=make)
    q = torch.randn(8 * 26, 8 * group, d, device="cuda", dtype=torch.bfloat16)
    if make is _infinite:  # (no product of zero and infinity, which is NaN)
        q = q.sign() * q.abs().clamp(min=0.1)
    if make is _tiny:
        q = q * 2.0 ** -50
    _check(c, q.to(torch.bfloat16), None, count, 1, 1)


def test_select_few_pages_for_many_tokens_of_chunks():
    c = Boxes([900, 300, 1400, 50], 16, 64, 16)
    q = torch.randn(127, 32, 64, device="cuda", dtype=torch.bfloat16)
    _check(c, q, [60, 30, 30, 5], 8, 0, 2)


def test_select_of_zero_queries():
    c = Boxes([5000], 2, 128, 16)
    q = torch.zeros(1, 8, 128, device="cuda", dtype=torch.bfloat16)
    _check(c, q, None, 30, 0, 1)
    q[0, 5] = 1.0
    _check(c, q, None, 30, 0, 1)


@pytest.mark.parametrize("bound", [math.nan, math.inf])
def test_select_of_zero_queries_and_infinite_bounds(bound):
    """Zero times an infinity is NaN, and above all."""
    def make(c):
        c.bounds[c.ids[0][17], :, 1, 5] = bound
    c = Boxes([5000], 2, 128, 16, make=make)
    q = torch.zeros(1, 8, 128, device="cuda", dtype=torch.bfloat16)
    pages = _check(c, q, None, 30, 0, 1)
    assert bool((pages == c.ids[0][17]).any(-1).all())


@pytest.mark.parametrize("explicit", [False, True])
def test_attention_of_padding_tokens(explicit):
    """Tokens behind the last sequence: a list that the call allocates holds no keys."""
    c = Boxes([700, 300], 2, 64, 16)
    q = torch.randn(40, 4, 64, device="cuda", dtype=torch.bfloat16)
    cache = c.handle
    cache.k.normal_()
    for _ in range(3):   # what the allocator hands out again
        x = [torch.full((40,), 1 << 28, device="cuda", dtype=torch.int32) for _ in range(8)]
        del x
        given = dict(lens=torch.zeros(40, device="cuda", dtype=torch.int32)) if explicit else {}
        pages, lens = _binding().paged_select(cache, q, c.bounds, c.table, c.kv_lens, 9,
                                              cu_seqlens=torch.tensor([0, 20, 30], device="cuda", dtype=torch.int32), **given)
        assert bool((lens[30:] == 0).all()) and bool((lens[:30] > 0).all())
        o, lse = _binding().paged_decode(cache, q, pages, lens)
        assert bool((o[30:] == 0).all()) and bool((lse[30:] == -math.inf).all())
        assert bool(torch.isfinite(o[:30].float()).all())
    _ok()


def test_select_many_equal_and_a_border_inside():
    """More than 512 pages at the border, equal in groups: ranked by digits."""
    def make(c):
        n = c.bounds.shape[0]
        c.bounds[:] = c.bounds[:1]
        c.bounds[..., 1] = (2 + torch.arange(n, device="cuda") % 3 / 64).to(torch.bfloat16)[:, None, None]
    c = Boxes([16 * 4000], 2, 64, 16, make=make)
    q = (torch.randn(1, 4, 64, device="cuda") * 8).to(torch.bfloat16)
    q[:, :, 1] = 2.0 ** -9   # differences far below the bound of a 32-bit sum's error
    _check(c, q, None, 900, 1, 1)
    c = Boxes([16 * 4000] * 50, 2, 64, 16, make=make)
    _check(c, q.expand(50, -1, -1).contiguous(), None, 900, 1, 1)


def test_select_bad_pages():
    c = Boxes([5000], 1, 64, 16)
    c.table[0, 5] = 10 ** 6
    q = torch.randn(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    pages, lens = _binding().paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, 20)
    assert _binding().attn_check(None) == 13
    assert bool(((pages >= 0) & (pages < c.bounds.shape[0])).all()) and int(lens) == 5000 - (313 - 20) * 16
    c.kv_lens.fill_(10 ** 7)
    _binding().paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, 20)
    assert _binding().attn_check(None) == 13


# ---------------------------------------------------------------- attention over lists

@pytest.mark.parametrize("kind", ["bf16", "e4m3", "pages"])
@pytest.mark.parametrize("B,H_kv,group,d,page,count", [
    (1, 1, 1, 64, 16, 1), (3, 2, 4, 128, 16, 5), (2, 8, 4, 128, 32, 64), (40, 2, 16, 64, 64, 9), (5, 3, 20, 128, 128, 3),
    (1, 8, 4, 128, 64, 200)])
def test_lists(B, H_kv, group, d, page, count, kind):
    n_pages = max(2 * count, 8)
    c = _make(kind, [n_pages * page], H_kv, d, page, seed=B)
    g = torch.Generator(device="cuda").manual_seed(B)
    at = torch.stack([torch.randperm(n_pages, generator=g, device="cuda")[:count] for _ in range(B * H_kv)]).view(B, H_kv, count)
    lists = torch.tensor(c.ids[0], device="cuda", dtype=torch.int32)[at].contiguous()
    lens = [(count - 1) * page + 1 + (7 * b) % page for b in range(B)]
    lens[-1] = 0 if B > 2 else lens[-1]
    lists[-1, :, lens[-1] // page + 1:] = -1
    kv_lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
    q = torch.randn(B, H_kv * group, d, device="cuda", dtype=torch.bfloat16)
    o, lse = _binding().paged_decode(c.handle(), q, lists, kv_lens)
    _ok()
    for b in range(B):
        n = lens[b]
        k, v = [], []
        for h in range(H_kv):
            ids = lists[b, h, :-(-n // page)].long()
            for out, name in ((k, "k"), (v, "v")):
                x = getattr(c, name)[:, h]
                x = as_int(x)[ids].view(x.dtype).double()
                if kind == "pages":
                    x = torch.ldexp(x, getattr(c, name + "_exp")[ids, h].double()[:, None, None] - 127)
                elif kind == "e4m3":
                    x = x * getattr(c, name + "_scale")[h].double()
                out.append(x.reshape(-1, d)[:n])
        want, want_abs, want_lse = attention(q[b:b + 1], torch.stack(k, 1), torch.stack(v, 1), 1 / math.sqrt(d),
                                             torch.tensor([n], device="cuda"))
        assert_attention(o[b:b + 1], lse[b][:, None], want, want_abs, want_lse, b)
    # any strides between the lists, given outputs, and the calls made from Python
    wide = torch.full((H_kv, B, count + 3), -1, device="cuda", dtype=torch.int32)
    wide[:, :, :count] = lists.transpose(0, 1)
    view = wide.transpose(0, 1)[:, :, :count]
    again = _binding().paged_decode(c.handle(), q, view, kv_lens, out=torch.empty_like(q))
    assert torch.equal(as_int(again[0]), as_int(o)) and torch.equal(again[1], lse)


def test_equal_lists_give_the_bits_of_a_page_table():
    c = Cache([5000, 100], 4, 128, 32, seed=3)
    q = torch.randn(2, 16, 128, device="cuda", dtype=torch.bfloat16)
    o, lse = _binding().paged_decode(c.handle(), q, c.table, c.kv_lens)
    lists = c.table[:, None].expand(-1, 4, -1).contiguous()
    o2, lse2 = _binding().paged_decode(c.handle(), q, lists, c.kv_lens)
    assert torch.equal(as_int(o), as_int(o2)) and torch.equal(lse, lse2)


def test_lists_bad_pages():
    c = Cache([500], 2, 64, 16, seed=3)
    q = torch.randn(1, 4, 64, device="cuda", dtype=torch.bfloat16)
    lists = c.table[:, None].expand(-1, 2, -1).contiguous()
    lists[0, 1, 3] = -1
    _binding().paged_decode(c.handle(), q, lists, c.kv_lens)
    assert _binding().attn_check(None) == 13


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kind", ["bf16", "pages"])
@pytest.mark.parametrize("drafted", [1, 3])
def test_decoding_with_selected_pages(kind, drafted):
    """Steps of a batch as a server makes them, captured once and replayed: append, bounds, selection,
    attention over the chosen pages. Each step against the definition over the pages that its
    own bounds choose."""
    B_ = _binding()
    H_kv, group, d, page, count, steps = 2, 4, 64, 16, 6, 20
    start = [40, 1, 160, 300]
    n = len(start)
    c = _make(kind, [x + steps * drafted for x in start], H_kv, d, page, seed=1)
    cache = c.handle()
    bounds = torch.zeros(c.k.shape[0], H_kv, 2, d, device="cuda", dtype=torch.bfloat16)
    kv_lens = torch.tensor(start, device="cuda", dtype=torch.int32)
    B_.paged_bounds(cache, bounds, c.table, kv_lens, cu_seqlens=_cu(start), tokens=sum(start))
    freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") * 2 / d)
    cu = None if drafted == 1 else _cu([drafted] * n)
    x = torch.zeros(n * drafted, H_kv * (group + 2), d, device="cuda", dtype=torch.bfloat16)

    def step():
        kv_lens.add_(drafted)
        q = B_.paged_append(cache, x[:, :-2 * H_kv], x[:, -2 * H_kv:-H_kv], x[:, -H_kv:], c.table, kv_lens, cu_seqlens=cu, inv_freq=freq)
        B_.paged_bounds(cache, bounds, c.table, kv_lens, cu_seqlens=cu, tokens=n * drafted)
        pages, lens = B_.paged_select(cache, q, bounds, c.table, kv_lens, count, cu_seqlens=cu, keep_first=1, keep_last=2)
        return q, pages, lens, *B_.paged_decode(cache, q, pages, lens)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    state = {m: getattr(c, m).clone() for m in (("k", "v", "k_exp", "v_exp") if kind == "pages" else ("k", "v"))}
    with torch.cuda.stream(stream):
        step()  # (attributes are set outside the capture)
        kv_lens.sub_(drafted)
        for m, t in state.items():
            as_int(getattr(c, m)).copy_(as_int(t))
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, pages, lens, o, lse = step()
    for i in range(steps):
        x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        _ok()
        for b in range(n):
            for j in range(drafted):
                t = b * drafted + j
                seen = start[b] + i * drafted + j + 1
                want_pages, keys = selected(q[t].view(H_kv, group, d), bounds, c.ids[b], seen, page, count, 1, 2)
                assert torch.equal(pages[t].cpu(), want_pages) and int(lens[t]) == keys
                if b != i % n:
                    continue
                k, v = [], []
                for h in range(H_kv):
                    ids = pages[t, h, :-(-keys // page)].long()
                    for out, name in ((k, "k"), (v, "v")):
                        y = as_int(getattr(c, name)[:, h])[ids].view(c.k.dtype).double()
                        if kind == "pages":
                            y = torch.ldexp(y, getattr(c, name + "_exp")[ids, h].double()[:, None, None] - 127)
                        out.append(y.reshape(-1, d)[:keys])
                want, want_abs, want_lse = attention(q[t:t + 1], torch.stack(k, 1), torch.stack(v, 1), 1 / math.sqrt(d),
                                                     torch.tensor([keys], device="cuda"))
                assert_attention(o[t:t + 1], lse[t][:, None], want, want_abs, want_lse, (i, b, j))
    # the bounds are those of the keys
    for b in range(n):
        total = start[b] + steps * drafted
        for i, p in enumerate(c.ids[b]):
            want = bounds_of(_keys(c, kind, p), min(page, total - i * page)).float().to(torch.bfloat16)
            assert torch.equal(bounds[p], want), (b, i)


def test_prompts_and_steps_captured_on_two_streams():
    """Whole prompts (the appending kernel by rows, chunk attention) and a selecting step over long tables
    (clusters), captured and replayed on two streams at once: the bits of eager calls."""
    B_ = _binding()
    H_kv, group, d, page = 2, 4, 128, 32
    new = [300, 70, 500]
    freq = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") * 2 / d)

    def world(seed):
        c = Pages([n + 1 for n in new], H_kv, d, page, seed=seed)
        cache = c.handle()
        c.kv_lens.sub_(1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(sum(new), H_kv * (group + 2), d, generator=g, device="cuda", dtype=torch.bfloat16)
        y = torch.randn(len(new), H_kv * (group + 2), d, generator=g, device="cuda", dtype=torch.bfloat16)
        bounds = torch.zeros(c.k.shape[0], H_kv, 2, d, device="cuda", dtype=torch.bfloat16)
        wide = torch.zeros(len(new), 3000, dtype=torch.int32, device="cuda")
        wide[:, :c.table.shape[1]] = c.table
        after, cu = c.kv_lens + 1, _cu(new)

        def work():
            q = B_.paged_append(cache, x[:, :-2 * H_kv], x[:, -2 * H_kv:-H_kv], x[:, -H_kv:], c.table, c.kv_lens, cu_seqlens=cu,
                                inv_freq=freq)
            B_.paged_bounds(cache, bounds, c.table, c.kv_lens, cu_seqlens=cu, tokens=sum(new))
            o, lse = B_.paged_forward(cache, q, c.table, c.kv_lens, cu)
            q1 = B_.paged_append(cache, y[:, :-2 * H_kv], y[:, -2 * H_kv:-H_kv], y[:, -H_kv:], wide, after, inv_freq=freq)
            B_.paged_bounds(cache, bounds, wide, after)
            pages, lens = B_.paged_select(cache, q1, bounds, wide, after, 5, keep_first=1)
            return (q, o, lse, q1, pages, lens, *B_.paged_decode(cache, q1, pages, lens))

        keep = (c, cache, x, y, bounds, wide, after, cu)
        return work, (c.k, c.v, c.k_exp, c.v_exp, bounds), keep

    worlds = [world(1), world(2)]
    eager = []
    for work, state, _ in worlds:
        out = work()
        eager.append([as_int(t).clone() if t.element_size() < 4 else t.clone() for t in (*out, *state)])
    _ok()
    streams = [torch.cuda.Stream() for _ in worlds]
    graphs, outs = [], []
    for (work, _, _), stream in zip(worlds, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(work())
        graphs.append(graph)
    for _ in range(5):
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    _ok()
    for out, (_, state, _), want in zip(outs, worlds, eager):
        for t, w in zip((*out, *state), want):
            assert torch.equal(as_int(t) if t.element_size() < 4 else t, w)


def test_pages_behind_2_31_elements():
    """Pages, lists and bounds whose places pass 32 bits."""
    B_ = _binding()
    H_kv, d, page = 8, 128, 256
    n_pages = (1 << 31) // (H_kv * page * d) + 6
    k = torch.empty(n_pages, H_kv, page, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.empty_like(k)
    exps = [torch.empty(n_pages, H_kv, dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = B_.PagedCache(k, v, k_scale=exps[0].view(torch.float8_e8m0fnu), v_scale=exps[1].view(torch.float8_e8m0fnu))
    bounds = torch.empty(n_pages, H_kv, 2, d, dtype=torch.bfloat16, device="cuda")
    ids = [n_pages - 1, 3, n_pages - 2, n_pages - 3]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    n = 3 * page + 40
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = torch.randn(n, 2 * H_kv, d, device="cuda", dtype=torch.bfloat16)
    B_.paged_append(cache, None, x[:, :H_kv], x[:, H_kv:], table, lens, cu_seqlens=_cu([n]))
    B_.paged_bounds(cache, bounds, table, lens, cu_seqlens=_cu([n]), tokens=n)
    q = torch.randn(1, 2 * H_kv, d, device="cuda", dtype=torch.bfloat16)
    pages, chosen = B_.paged_select(cache, q, bounds, table, lens, 3, keep_first=1)
    o, lse = B_.paged_decode(cache, q, pages, chosen)
    full, full_lse = B_.paged_decode(cache, q, table, lens)
    _ok()
    values = [values_of(t[ids], e[ids]) for t, e in ((k, exps[0]), (v, exps[1]))]  # [4, H_kv, page, d]
    for i in range(4):
        rows = min(page, n - i * page)
        assert torch.equal(bounds[ids[i]], bounds_of(values[0][i], rows).float().to(torch.bfloat16))
    want, keys = selected(q[0].view(H_kv, 2, d), bounds, ids, n, page, 3, 1, 1)
    assert torch.equal(pages[0].cpu(), want) and int(chosen) == keys
    place = {p: i for i, p in enumerate(ids)}
    for lists, length, got, got_lse in ((pages, keys, o, lse), (table[:, None].expand(-1, H_kv, -1), n, full, full_lse)):
        kv = [torch.stack([torch.cat([t[place[int(p)], h] for p in lists[0, h]])[:length] for h in range(H_kv)], 1) for t in values]
        want, want_abs, want_lse = attention(q, *kv, 1 / math.sqrt(d), torch.tensor([length], device="cuda"))
        assert_attention(got, got_lse[0][:, None], want, want_abs, want_lse, length)


def test_selection_is_the_same_again_and_on_another_stream():
    c = Boxes([50000] * 3, 4, 128, 16, seed=5)
    q = torch.randn(3, 16, 128, device="cuda", dtype=torch.bfloat16)
    pages, lens = _binding().paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, 100)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    out = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            out.append(_binding().paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, 100))
    torch.cuda.synchronize()
    for p, n in out:
        assert torch.equal(p, pages) and torch.equal(n, lens)
    _ok()


def test_offsets_that_are_no_offsets_stay_inside():
    """Decreasing, overlapping and negative offsets write nothing outside and are recorded."""
    B_ = _binding()
    c = Pages([200, 300, 100], 2, 64, 16, seed=3)
    guard = torch.randint(0, 255, (64, 2, 16, 64), dtype=torch.uint8, device="cuda")
    before = guard.clone()
    bounds = torch.zeros(c.k.shape[0], 2, 2, 64, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(120, 2, 64, device="cuda", dtype=torch.bfloat16)
    for bad in ([0, 90, 40, 120], [5, 60, 90, 120], [0, -7, 60, 500], [100, 50, 20, 10]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        q = torch.randn(120, 4, 64, device="cuda", dtype=torch.bfloat16)
        B_.paged_append(c.handle(), q, x, x, c.table, c.kv_lens, cu_seqlens=cu)
        B_.paged_bounds(c.handle(), bounds, c.table, c.kv_lens, cu_seqlens=cu, tokens=120)
        pages, _ = B_.paged_select(c.handle(), q, bounds, c.table, c.kv_lens, 4, cu_seqlens=cu)
        assert B_.attn_check(None) == 12
        assert torch.equal(guard, before)
