"""The paged key-value cache on the GPU: appending with the rotary embedding,
one-token attention and chunk attention, against definitions in 64 bits, and a
run of all of them as a serving loop makes it."""

import ctypes
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from paged_common import (BF16, E4M3, E4M3_MAX, Cache, as_int, assert_attention, attention,  # noqa: E402
                          turned)

PAGES_ERR, SEQLENS_ERR = 13, 12


@pytest.fixture(autouse=True)
def _clean():
    assert binding.attn_check(None) == 0
    yield
    assert binding.attn_check(None) == 0


def _q(n, H_q, d, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, H_q, d, generator=g, device="cuda").to(torch.bfloat16)


def _table(c, tokens):
    """The page table, or one that could hold that many tokens a sequence: what a table
    can hold decides which kernel a call of little work runs on (clusters, dealt-out
    units, the tensor cores)."""
    if not tokens:
        return c.table
    table = torch.full((len(c.lens), max(c.width, tokens // c.page)), -7, dtype=torch.int32, device="cuda")
    table[:, :c.width] = c.table
    return table


def _decode_want(c, q, scale):
    parts = [attention(q[b:b + 1], c.keys[b], c.values[b], scale, torch.tensor([n], device="cuda"))
             for b, n in enumerate(c.lens)]
    return (torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]),
            torch.stack([p[2][:, 0] for p in parts]))


DECODE = [
    # lens, H_q, H_kv, d, page
    ([1], 1, 1, 64, 16),
    ([0], 4, 2, 128, 16),
    ([0, 5, 0, 64, 63, 65, 0], 8, 2, 128, 16),
    ([1, 2, 3, 15, 16, 17, 31, 33], 8, 8, 64, 16),
    ([128, 127, 129, 255, 256, 257], 16, 2, 128, 32),
    ([700], 32, 8, 128, 64),
    ([40000], 8, 1, 128, 128),
    ([9000, 1, 3000, 0, 77], 10, 2, 128, 256),
    ([513, 2000], 14, 2, 64, 32),
    ([300, 50], 16, 1, 128, 16),
    ([300, 1000], 48, 2, 64, 128),
    ([129, 640], 34, 1, 128, 64),
    (list(range(0, 330)), 4, 2, 64, 16),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(DECODE)))
def test_decode(case, kind):
    lens, H_q, H_kv, d, page = DECODE[case]
    c = Cache(lens, H_kv, d, page, kind, seed=case)
    q = _q(len(lens), H_q, d)
    for scale in (1.0 / math.sqrt(d), -0.03):
        o, lse = binding.paged_decode(c.handle(), q, c.table, c.kv_lens, scale=scale)
        assert_attention(o, lse, *_decode_want(c, q, scale), what=scale)


SHORT = [
    # lens, H_q, H_kv, d, page
    ([777], 32, 8, 128, 16),
    ([0, 1, 64, 65, 127, 129, 2048, 500], 4, 1, 128, 64),
    ([512, 0, 511, 63, 64, 65, 1, 300], 32, 8, 128, 16),
    ([1, 40, 0, 128, 129, 500, 512, 448] * 2, 16, 8, 128, 32),
    ([512, 1, 2, 64, 65, 300, 0, 449] * 4, 8, 8, 64, 16),
    ([1000, 200, 0, 64], 40, 1, 64, 256),  # three chunks of 16 query rows
    ([4096], 16, 2, 128, 128),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(SHORT)))
def test_decode_of_short_and_of_wide_tables(case, kind):
    """A table that holds little sends a call to clusters that share a (sequence, KV
    head) each; the same sequences in a wide table are dealt out to all CTAs."""
    lens, H_q, H_kv, d, page = SHORT[case]
    c = Cache(lens, H_kv, d, page, kind, seed=case)
    h, q = c.handle(), _q(len(lens), H_q, d)
    want = _decode_want(c, q, 1.0 / math.sqrt(d))
    for table in (c.table, _table(c, 100000)):
        o, lse = binding.paged_decode(h, q, table, c.kv_lens)
        assert_attention(o, lse, *want, what=tuple(table.shape))
        again = binding.paged_decode(h, q, table, c.kv_lens)
        assert torch.equal(as_int(o), as_int(again[0])) and torch.equal(lse, again[1])


def test_short_decode_captured():
    """A captured short call replays with other lengths, none of them among these, and
    with an infinite score, which the sequence's own output alone shows."""
    c = Cache([600, 17, 0, 450], 2, 128, 32, width=20)
    h, q = c.handle(), _q(4, 8, 128)
    graph = torch.cuda.CUDAGraph()
    binding.paged_decode(h, q, c.table, c.kv_lens)
    with torch.cuda.graph(graph):
        o, lse = binding.paged_decode(h, q, c.table, c.kv_lens)
    for lens in ([600, 17, 0, 450], [1, 0, 0, 449], [64, 16, 0, 65], [0, 0, 0, 0]):
        c.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        cut = Cache.__new__(Cache)
        cut.lens = lens
        cut.keys = [x[:n] for x, n in zip(c.keys, lens)]
        cut.values = [x[:n] for x, n in zip(c.values, lens)]
        assert_attention(o, lse, *_decode_want(cut, q, 1.0 / math.sqrt(128)), what=lens)
    c.kv_lens.copy_(torch.tensor([600, 17, 0, 450], dtype=torch.int32))
    c.put(c.k, 0, 599, torch.full((1, 2, 128), math.inf, dtype=torch.bfloat16, device="cuda"))
    graph.replay()
    assert not bool(torch.isfinite(lse[0]).any())
    want = _decode_want(c, q, 1.0 / math.sqrt(128))
    assert_attention(o[1:], lse[1:], *(x[1:] for x in want))


def test_decode_is_bit_exact_and_captured():
    """Two calls give the same bits; a captured call replays with new contents,
    lengths and pages, in its own outputs and workspace."""
    c = Cache([3000, 17, 0, 450], 4, 128, 32, width=120)
    h, q = c.handle(), _q(4, 16, 128)
    a = binding.paged_decode(h, q, c.table, c.kv_lens)
    b = binding.paged_decode(h, q, c.table, c.kv_lens)
    assert all(torch.equal(as_int(x.view(torch.int16)), as_int(y.view(torch.int16))) for x, y in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = binding.paged_decode(h, q, c.table, c.kv_lens)
    graph.replay()
    assert torch.equal(o, a[0]) and torch.equal(lse, a[1])
    q.copy_(_q(4, 16, 128, seed=9))
    c.lens = [2999, 1, 0, 200]
    c.kv_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    graph.replay()
    c.keys = [x[:n] for x, n in zip(c.keys, c.lens)]
    c.values = [x[:n] for x, n in zip(c.values, c.lens)]
    assert_attention(o, lse, *_decode_want(c, q, 1.0 / math.sqrt(128)))


def test_decode_layouts_streams_and_given_buffers():
    """Keys and values as halves of one tensor, a page table that is a slice of a
    wider one, another stream, caller's outputs and workspace."""
    c = Cache([130, 1, 77], 2, 64, 16, paired=True)
    q = _q(3, 6, 64)
    wide = torch.full((3, c.width + 5), 99999, dtype=torch.int32, device="cuda")
    wide[:, :c.width] = c.table
    out = torch.empty_like(q)
    lse = torch.empty(3, 6, device="cuda")
    ws = torch.full((binding.paged_workspace_bytes(c.handle(), 6),), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = binding.paged_decode(c.handle(), q, wide[:, :c.width], c.kv_lens, out=out, lse=lse, workspace=ws)
    s.synchronize()
    assert got[0] is out and got[1] is lse
    assert_attention(out, lse, *_decode_want(c, q, 1.0 / 8.0))


def test_decode_large_query_values_over_e4m3():
    """Query rows far outside fp16's range: a power of two brings them into it."""
    c = Cache([100, 300], 2, 128, 16, "e4m3")
    for factor in (2.0 ** 40, 2.0 ** -60):
        q = (_q(2, 8, 128).float() * factor).to(torch.bfloat16)
        scale = 1.0 / math.sqrt(128) / factor
        o, lse = binding.paged_decode(c.handle(), q, c.table, c.kv_lens, scale=scale)
        assert_attention(o, lse, *_decode_want(c, q, scale), what=factor)


@pytest.mark.parametrize("wide", [0, 100000])
def test_chunk_large_query_values_over_e4m3(wide):
    """The same in the tensor-core kernel's fp16 queries, and given buffers."""
    c = Cache([300, 200], 2, 128, 16, "e4m3")
    new, h = [150, 200], c.handle()
    ws = torch.full((binding.paged_workspace_bytes(h, 8, 350, 2),), 255, dtype=torch.uint8, device="cuda")
    for factor in (2.0 ** 40, 2.0 ** -60):
        q = (_q(350, 8, 128).float() * factor).to(torch.bfloat16)
        scale = 1.0 / math.sqrt(128) / factor
        o, lse = binding.paged_forward(h, q, _table(c, wide), c.kv_lens, _offsets(new), scale=scale, workspace=ws)
        assert_attention(o, lse, *_chunk_want(c, q, new, scale, True), what=factor)


@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("wide", [0, 100000])
def test_small_weights_over_e4m3(wide, n):
    """A key with weight 1 and no value next to 199 with weights of 2^-19: they keep the
    accuracy of larger ones (as fp16 numbers of their own they would have 5 bits)."""
    c = Cache([200], 1, 128, 16, "e4m3")
    c.k_scale.fill_(0.25)
    c.v_scale.fill_(0.5)
    k = torch.zeros(200, 1, 128, device="cuda")
    k[0, 0, 0] = 4.0
    v = torch.randint(1, 8, (200, 1, 128), device="cuda").float()
    v[0] = 0.0
    for cache, x in ((c.k, k), (c.v, v)):
        c.put(cache, 0, 0, x.to(torch.float8_e4m3fn))
    c.keys, c.values = [k.double() * 0.25], [v.double() * 0.5]
    q = torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 19.0
    scale = math.log(2.0)
    if n == 1:
        o, lse = binding.paged_decode(c.handle(), q, _table(c, wide), c.kv_lens, scale=scale)
        want = _decode_want(c, q, scale)
    else:
        o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets([n]), scale=scale, causal=False)
        want = _chunk_want(c, q, [n], scale, False)
    assert_attention(o, lse, *want)


def test_decode_spread_scores():
    """Scores with a wide spread: the running maximum moves many times."""
    c = Cache([2000], 1, 64, 16)
    ramp = torch.linspace(-60, 60, 2000, device="cuda")[torch.randperm(2000, device="cuda")]
    k = torch.zeros(2000, 1, 64, device="cuda")
    k[:, 0, 0] = ramp
    k = k.to(torch.bfloat16)
    c.put(c.k, 0, 0, k)
    c.keys = [k.double()]
    q = torch.zeros(1, 8, 64, device="cuda", dtype=torch.bfloat16)
    q[0, :, 0] = torch.tensor([1, 2, -1, 0.5, 0, 3, -2, 0.25])
    o, lse = binding.paged_decode(c.handle(), q, c.table, c.kv_lens, scale=1.0)
    assert_attention(o, lse, *_decode_want(c, q, 1.0))


CHUNK = [
    # new tokens, lens, H_q, H_kv, d, page
    ([1], [1], 2, 1, 64, 16),
    ([4, 4], [300, 64], 8, 2, 128, 16),
    ([5, 0, 1, 7], [5, 40, 1000, 133], 16, 2, 128, 32),
    ([3, 9], [1, 9], 4, 4, 64, 16),          # more rows than keys: padding
    ([2, 3], [0, 3], 4, 2, 128, 16),         # rows of a sequence without keys
    ([100], [100], 4, 4, 64, 16),
    ([129, 250, 1], [129, 700, 2], 8, 2, 128, 64),
    ([257, 130], [5000, 130], 10, 2, 128, 128),
    ([333], [2048], 7, 1, 64, 32),
    ([512, 64, 65], [512, 640, 8000], 4, 1, 128, 256),
    ([40], [3000], 24, 1, 128, 64),
    ([300, 20], [300, 20], 64, 1, 64, 16),
    ([6, 150], [70, 200], 200, 1, 64, 16),   # more heads on one KV head than a tile has rows
    ([2] * 300, list(range(2, 302)), 2, 2, 64, 16),
]


def _chunk_want(c, q, new, scale, causal):
    o, a, lse, t0 = [], [], [], 0
    for b, n in enumerate(new):
        L = c.lens[b]
        last = torch.full((n,), L, device="cuda")
        if causal:
            last = torch.clamp(L - n + 1 + torch.arange(n, device="cuda"), min=0)
        r = attention(q[t0:t0 + n], c.keys[b], c.values[b], scale, last)
        o.append(r[0]), a.append(r[1]), lse.append(r[2])
        t0 += n
    return torch.cat(o), torch.cat(a), torch.cat(lse, 1)


def _many(B, H_q, H_kv, d, page, new_lo, new_hi, ctx_hi, seed):
    """A larger ragged batch: new tokens, lengths and the rest of a CHUNK case."""
    r = random.Random(seed)
    new = [r.randint(new_lo, new_hi) for _ in range(B)]
    return new, [n + r.randint(0, ctx_hi) for n in new], H_q, H_kv, d, page


# the tensor-core kernel's ways of dealing out work: claimed tiles beyond the listed
# ones; whole waves and a rest that is cut; more sequences than are sorted
MANY = [
    _many(24, 16, 16, 64, 16, 257, 300, 200, 1),
    _many(10, 16, 16, 64, 32, 200, 256, 900, 2),
    _many(21, 32, 16, 64, 64, 65, 128, 40, 3),
    _many(1100, 4, 1, 64, 16, 0, 12, 30, 4),
    _many(1, 4, 4, 128, 64, 700, 700, 9000, 5),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(MANY)))
@pytest.mark.parametrize("wide", [0, 100000])
def test_chunk_of_many(wide, case, kind):
    new, lens, H_q, H_kv, d, page = MANY[case]
    c = Cache(lens, H_kv, d, page, kind, seed=case)
    q = _q(sum(new), H_q, d)
    table = _table(c, wide)
    o, lse = binding.paged_forward(c.handle(), q, table, c.kv_lens, _offsets(new))
    assert_attention(o, lse, *_chunk_want(c, q, new, 1.0 / math.sqrt(d), True))
    again = binding.paged_forward(c.handle(), q, table, c.kv_lens, _offsets(new))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_calls_on_two_streams_at_once():
    """Two streams, each with its own decoding and chunk calls over one cache: the
    same bits as one after the other (workspaces are the calls' own)."""
    c = Cache([5000, 300, 2000], 4, 128, 64)
    h, new = c.handle(), [40, 300, 129]  # (on the tensor cores)
    qs = [(_q(3, 16, 128, seed=i), _q(sum(new), 16, 128, seed=10 + i)) for i in range(2)]
    cu = _offsets(new)

    def calls(q1, qn):
        return [*binding.paged_decode(h, q1, c.table, c.kv_lens), *binding.paged_forward(h, qn, c.table, c.kv_lens, cu)]

    want = [calls(*q) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(*qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_behind_2_to_the_31_elements(kind):
    """Pages whose offsets need more than 32 bits, read and written."""
    H_kv, page, d = 8, 256, 128
    pages = (1 << 31) // (H_kv * page * d) + 40
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    k, v = (torch.empty(pages, H_kv, page, d, dtype=dtype, device="cuda") for _ in range(2))
    ids = [pages - 1, pages - 7, pages - 3]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([600], dtype=torch.int32, device="cuda")
    h, cu = binding.PagedCache(k, v), _offsets([600])
    new_k, new_v, q = _q(600, H_kv, d, 2), _q(600, H_kv, d, 3), _q(600, 16, d)
    binding.paged_append(h, None, new_k, new_v, table, lens, cu_seqlens=cu)
    stored = [torch.cat([t[i].transpose(0, 1) for i in ids])[:600].double() for t in (k, v)]
    if kind == "bf16":
        assert torch.equal(stored[0], new_k.double()) and torch.equal(stored[1], new_v.double())
    last = torch.arange(1, 601, device="cuda")
    o, lse = binding.paged_forward(h, q, table, lens, cu)
    assert_attention(o, lse, *attention(q, *stored, 1.0 / math.sqrt(d), last))
    o, lse = binding.paged_decode(h, q[599:], table, lens)
    want = attention(q[599:], *stored, 1.0 / math.sqrt(d), last[599:])
    assert_attention(o, lse, want[0], want[1], want[2].t())


def _offsets(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CHUNK)))
@pytest.mark.parametrize("wide", [0, 16000, 100000])
def test_chunk(wide, case, kind, causal):
    new, lens, H_q, H_kv, d, page = CHUNK[case]
    c = Cache(lens, H_kv, d, page, kind, seed=case)
    q = _q(sum(new), H_q, d)
    for scale in (1.0 / math.sqrt(d), -0.05):
        o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new), scale=scale,
                                       causal=causal)
        assert_attention(o, lse, *_chunk_want(c, q, new, scale, causal), what=scale)


@pytest.mark.parametrize("n", [3, 200])
@pytest.mark.parametrize("wide", [0, 100000])
def test_chunk_leaves_rows_behind_the_last_sequence(wide, n):
    new = [n, 2 * n]
    c = Cache([n, 500], 2, 128, 16)
    T = 3 * n + 50
    q = _q(T, 8, 128)
    out = torch.full_like(q, 7.0)
    lse = torch.full((8, T), 3.0, device="cuda")
    binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new), out=out, lse=lse)
    assert bool((out[3 * n:] == 7.0).all()) and bool((lse[:, 3 * n:] == 3.0).all())
    assert_attention(out[:3 * n], lse[:, :3 * n], *_chunk_want(c, q, new, 1.0 / math.sqrt(128), True))


@pytest.mark.parametrize("n", [2, 300])
@pytest.mark.parametrize("wide", [0, 100000])
def test_chunk_captured(wide, n):
    """A captured call replays over other lengths in the same buffers."""
    c = Cache([1000, 400], 2, 64, 16, width=70)
    h, q, cu, table = c.handle(), _q(2 * n, 4, 64), _offsets([n, n]), _table(c, wide)
    binding.paged_forward(h, q, table, c.kv_lens, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = binding.paged_forward(h, q, table, c.kv_lens, cu)
    c.lens = [999, 302]
    c.kv_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.keys = [x[:m] for x, m in zip(c.keys, c.lens)]
    c.values = [x[:m] for x, m in zip(c.values, c.lens)]
    new = [n, n]
    for _ in range(2):
        graph.replay()
        assert_attention(o, lse, *_chunk_want(c, q, new, 1.0 / 8.0, True))


@pytest.mark.parametrize("wide", [0, 100000])
def test_chunk_agrees_with_the_packed_forward(wide):
    """A fresh prompt through the cache gives what attn_fwd gives on its rows: both
    within bf16's rounding of P and of O of the same value."""
    new = [300, 129, 64]
    c = Cache(new, 2, 128, 16)
    q = _q(sum(new), 8, 128)
    o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new))
    k, v = (torch.cat([x.to(torch.bfloat16) for x in y]) for y in (c.keys, c.values))
    o2, lse2 = binding.forward(q, k, v, causal=True, cu_seqlens=_offsets(new))
    _, size, _ = _chunk_want(c, q, new, 1.0 / math.sqrt(128), True)
    bound = 2 * BF16 * o.double().abs() + 2 * (BF16 + 2.0 ** -12) * size
    assert bool(((o.double() - o2.double()).abs() <= bound).all())
    assert bool(((lse - lse2).abs() <= 2.0 ** -12 + 2.0 ** -21 * lse2.abs()).all())


APPEND = [
    # new tokens, lengths after, H_q, H_kv, d, page, rotary, interleaved
    ([1], [1], 1, 1, 64, 16, 64, False),
    ([1, 1, 1], [5, 1000001, 0], 8, 2, 128, 256, 128, False),   # far positions; a padded row
    ([1, 1], [17, 16], 4, 4, 128, 16, 128, True),
    ([33, 0, 100], [33, 7, 150], 10, 2, 64, 16, 32, True),
    ([5, 9], [3, 40], 4, 2, 128, 32, 64, False),                # more rows than positions
    ([70, 3], [128, 3], 6, 1, 128, 64, 16, False),
    ([20], [25], 0, 3, 64, 16, 48, True),
    ([300], [300], 32, 8, 128, 128, 0, False),
]


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append(case, kind, fused):
    new, lens, H_q, H_kv, d, page, rotary, inter = APPEND[case]
    far = max(lens) > 100000
    c = Cache(lens, H_kv, d, page, kind, seed=case) if not far else _far_cache(lens, H_kv, d, page, kind)
    T = sum(new)
    if fused:
        x = _q(T, H_q + 2 * H_kv, d)
        q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    else:
        q, k, v = _q(T, max(H_q, 1), d)[:, :H_q], _q(T, H_kv, d, 2), _q(T, H_kv, d, 3)
    freq = (10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / rotary)).cuda() if rotary else None
    cu = None if all(n == 1 for n in new) else _offsets(new)
    before = as_int(c.k).clone(), as_int(c.v).clone()
    q_out = torch.full((T, H_q, d), 5.0, dtype=torch.bfloat16, device="cuda") if H_q else None
    got = binding.paged_append(c.handle(), q if H_q else None, k, v, c.table, c.kv_lens, cu_seqlens=cu,
                               inv_freq=freq, interleaved=inter, q_out=q_out)
    assert got is q_out
    t0 = 0
    for b, n in enumerate(new):
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        rows = torch.arange(t0, t0 + n, device="cuda")
        t0 += n
        live = pos >= 0
        if H_q:
            assert bool((got[rows[~live]] == 5.0).all())
            want, size = turned(q[rows[live]].cpu(), pos[live].cpu(), None if freq is None else freq.cpu(), inter)
            err = (got[rows[live]].cpu().double() - want).abs()
            assert bool((err <= BF16 * want.abs() + 2.0 ** -20 * size).all())
        for cache, x, scale, was, fr in ((c.k, k, c.k_scale, before[0], freq), (c.v, v, c.v_scale, before[1], None)):
            m = int(live.sum())
            if m == 0:
                continue
            want, size = turned(x[rows[live]].cpu(), pos[live].cpu(), None if fr is None else fr.cpu(), inter)
            have = c.get(cache, b, int(pos[live][0]), m).cpu().double()
            if kind == "e4m3":
                s = scale.cpu().double()[:, None]
                want, size = want / s, size / s
                # below 2^-6 the steps are 2^-9 whatever the value
                bound = E4M3 * want.abs() + 2.0 ** -10 + 2.0 ** -18 * size
                big = want.abs() >= E4M3_MAX
                assert bool((have[big].abs() == E4M3_MAX).all())
                bound = torch.where(big, torch.full_like(bound, math.inf), bound)
            else:
                bound = BF16 * want.abs() + 2.0 ** -20 * size
            assert bool(((have - want).abs() <= bound).all())
            # mark the rows, to see below that nothing else changed
            c.put(cache, b, int(pos[live][0]), c.get(was.view(cache.dtype), b, int(pos[live][0]), m))
    assert torch.equal(as_int(c.k), before[0]) and torch.equal(as_int(c.v), before[1])


def _far_cache(lens, H_kv, d, page, kind):
    """Long sequences that own only the page of their last token."""
    c = Cache([0] * len(lens), H_kv, d, page, kind, spare=len(lens) + 1, width=-(-max(lens) // page))
    c.lens = lens
    for b, n in enumerate(lens):
        c.ids[b] = [b] * -(-n // page)
        if n:
            c.table[b, (n - 1) // page] = b
    c.kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return c


def test_append_in_place_and_without_rotation():
    c = Cache([40], 2, 64, 16)
    x = _q(40, 8, 64)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    was = q.clone()
    assert binding.paged_append(c.handle(), q, k, v, c.table, c.kv_lens, cu_seqlens=_offsets([40])) is q
    assert torch.equal(q, was) and torch.equal(c.get(c.k, 0, 0, 40), k) and torch.equal(c.get(c.v, 0, 0, 40), v)
    freq = (500.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    apart = binding.paged_append(c.handle(), q, k, v, c.table, c.kv_lens, cu_seqlens=_offsets([40]), inv_freq=freq)
    assert torch.equal(q, was)
    assert binding.paged_append(c.handle(), q, k, v, c.table, c.kv_lens, cu_seqlens=_offsets([40]), inv_freq=freq,
                                q_out=q) is q
    assert torch.equal(q, apart)


def test_append_nan_and_infinities_over_e4m3():
    c = Cache([2], 1, 64, 16, "e4m3")
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan])
    binding.paged_append(c.handle(), None, k, k, c.table, c.kv_lens, cu_seqlens=_offsets([2]))
    got = c.get(c.v, 0, 0, 2).float()
    assert got[0, 0, 0] == E4M3_MAX and got[0, 0, 1] == -E4M3_MAX and got[0, 0, 2].isnan()
    assert bool((got.flatten()[3:] == 0).all())


@pytest.mark.parametrize("what", ["page", "length", "offsets"])
def test_bad_arrays_stay_inside_and_are_reported(what):
    """Pages outside the cache, lengths past the page table and decreasing offsets:
    nothing outside is read or written (a guard page after the cache keeps its
    contents), the call reports it, the next call works."""
    H_kv, d, page = 2, 64, 16
    c = Cache([40, 30], H_kv, d, page, spare=3)
    guard = torch.full((c.k.shape[0] + 2, H_kv, page, d), 9.0, dtype=torch.bfloat16, device="cuda")
    k, v = guard.clone(), guard.clone()
    inner = slice(1, 1 + c.k.shape[0])
    k[inner], v[inner] = c.k, c.v
    h = binding.PagedCache(k[inner], v[inner])
    table, lens, cu = c.table.clone(), c.kv_lens.clone(), _offsets([3, 4])
    if what == "page":
        table[0, 2], table[1, 1] = 1 << 30, -1
    elif what == "length":
        lens = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
        table = table.clamp(min=0)
    else:
        cu = torch.tensor([0, 5, 2], dtype=torch.int32, device="cuda")
    x = _q(7, 4, d)
    binding.paged_append(h, x[:, :2], x[:, :2], x[:, 2:], table, lens, cu_seqlens=cu)
    expect = SEQLENS_ERR if what == "offsets" else PAGES_ERR
    assert binding.attn_check(None) == expect
    binding.paged_forward(h, x, table, lens, cu)
    assert binding.attn_check(None) == expect
    if what != "offsets":
        binding.paged_decode(h, x[:2].contiguous(), table, lens)
        assert binding.attn_check(None) == expect
    for t in (k, v):
        assert bool((t[0] == 9.0).all()) and bool((t[-1] == 9.0).all())
    q = _q(2, 4, d)
    c2 = Cache([40, 30], H_kv, d, page)
    o, lse = binding.paged_decode(c2.handle(), q, c2.table, c2.kv_lens)
    assert_attention(o, lse, *_decode_want(c2, q, 1.0 / 8.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_serving_loop(kind):
    """Prompts appended and answered, then tokens one by one: at every step the
    outputs are those of the definition over what the cache was given, and a
    captured step replays with the lengths and tokens of the moment."""
    H_q, H_kv, d, page = 8, 2, 64, 16
    new = [37, 5, 160]
    c = Cache(new, H_kv, d, page, kind, spare=12, width=14)
    free = sorted(set(range(c.k.shape[0])) - {i for ids in c.ids for i in ids})
    freq = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) * 2 / d)).cuda()
    h, scale = c.handle(), 1.0 / math.sqrt(d)
    x = _q(sum(new), H_q + 2 * H_kv, d, seed=5)

    def remember(rows, b, start):
        """The cache's own rows, in 64 bits (its rounding has a test of its own)."""
        for cache, sc, kept in ((c.k, c.k_scale, c.keys), (c.v, c.v_scale, c.values)):
            y = c.get(cache, b, start, rows).double()
            y = y if sc is None else y * sc.double()[:, None]
            kept[b] = torch.cat((kept[b][:start], y))

    q = binding.paged_append(h, x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:], c.table, c.kv_lens,
                             cu_seqlens=_offsets(new), inv_freq=freq)
    for b, n in enumerate(new):
        remember(n, b, 0)
    o, lse = binding.paged_forward(h, q, c.table, c.kv_lens, _offsets(new))
    assert_attention(o, lse, *_chunk_want(c, q, new, scale, True))

    step_x = torch.empty(3, H_q + 2 * H_kv, d, dtype=torch.bfloat16, device="cuda")

    def step():
        q = binding.paged_append(h, step_x[:, :H_q], step_x[:, H_q:H_q + H_kv], step_x[:, H_q + H_kv:], c.table,
                                 c.kv_lens, inv_freq=freq)
        return (q, *binding.paged_decode(h, q, c.table, c.kv_lens))

    def advance(i):
        for b in range(3):
            if c.lens[b] % page == 0:
                c.ids[b].append(free.pop())
                c.table[b, len(c.ids[b]) - 1] = c.ids[b][-1]
            c.lens[b] += 1
        c.kv_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        step_x.copy_(_q(3, H_q + 2 * H_kv, d, seed=100 + i))

    def check(q, o, lse):
        for b in range(3):
            remember(1, b, c.lens[b] - 1)
        assert_attention(o, lse, *_decode_want(c, q, scale))

    advance(0)
    check(*step())
    graph = torch.cuda.CUDAGraph()
    advance(1)
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(2, 14):
        graph.replay()
        check(*outs)
        advance(i)


def test_compiled_calls_and_python_checks_agree():
    """The calls that allocate their outputs are checked and made in C, those with
    given outputs in Python: the same bits, the same refusals."""
    c = Cache([40, 30], 2, 64, 16)
    h, q, cu = c.handle(), _q(2, 4, 64), _offsets([1, 1])
    for call in (lambda **kw: binding.paged_decode(h, q, c.table, c.kv_lens, **kw),
                 lambda **kw: binding.paged_forward(h, q, c.table, c.kv_lens, cu, **kw)):
        a = call()
        b = call(out=torch.empty_like(q), lse=torch.empty_like(a[1]))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    k, freq = _q(2, 2, 64), torch.ones(32, dtype=torch.float64, device="cuda")
    bad = [
        lambda: binding.paged_decode(h, q.float(), c.table, c.kv_lens),
        lambda: binding.paged_decode(h, q.cpu(), c.table, c.kv_lens),
        lambda: binding.paged_decode(h, _q(3, 4, 64), c.table, c.kv_lens),
        lambda: binding.paged_decode(h, _q(2, 3, 64), c.table, c.kv_lens),
        lambda: binding.paged_decode(h, _q(2, 4, 128), c.table, c.kv_lens),
        lambda: binding.paged_decode(h, _q(2, 8, 64)[:, :4], c.table, c.kv_lens),
        lambda: binding.paged_decode(h, q, c.table.long(), c.kv_lens),
        lambda: binding.paged_decode(h, q, c.table[:1], c.kv_lens),
        lambda: binding.paged_decode(h, q, c.table, c.kv_lens.cpu()),
        lambda: binding.paged_forward(h, q, c.table, c.kv_lens, cu[:2]),
        lambda: binding.paged_forward(h, q, c.table, c.kv_lens, None),
        lambda: binding.paged_append(h, q, _q(2, 1, 64), k, c.table, c.kv_lens),
        lambda: binding.paged_append(h, q, k, _q(3, 2, 64), c.table, c.kv_lens),
        lambda: binding.paged_append(h, _q(1, 4, 64), k, k, c.table, c.kv_lens),
        lambda: binding.paged_append(h, q, k, k, c.table, c.kv_lens, inv_freq=freq.float()),
        lambda: binding.paged_append(h, q, k, k, c.table, c.kv_lens, q_out=_q(2, 2, 64)),
        lambda: binding.paged_append(h, None, k, k, c.table, c.kv_lens, q_out=q),
        lambda: binding.PagedCache(c.k, c.v, k_scale=torch.ones(2, device="cuda")),
        lambda: binding.PagedCache(c.k.transpose(1, 2), c.v.transpose(1, 2)),
        lambda: binding.PagedCache(c.k, c.v[:1]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: binding.paged_append(h, q, k, k, c.table, c.kv_lens, inv_freq=freq[:4]),  # 8 elements
              lambda: binding.paged_decode(h, q, c.table, c.kv_lens, scale=float("nan"))):
        with pytest.raises(binding.AttnError) as e:
            f()
        assert e.value.status == 4
    with pytest.raises(ctypes.ArgumentError):
        binding.paged_decode(h, q, c.table, c.kv_lens, scale="1")


def test_append_divides_by_the_scale_exactly():
    """e4m3 values are those of the 32-bit quotient, rounded to nearest: on scales of
    many mantissas, on quotients at and next to the borders between two of e4m3's
    values, and with scales outside the normal range of a rounded inverse."""
    g = torch.Generator(device="cuda").manual_seed(3)
    H_kv, d, n = 8, 64, 512
    c = Cache([n], H_kv, d, 64, "e4m3")
    grid = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()  # 0 .. 448
    border = (grid[1:] + grid[:-1]) / 2
    for mantissa in ([1.0] * H_kv, None, [1e-38, 3e-39, 2e38, 1e-31, 1e31, 1.5, 1.9999999, 1.0000001]):
        if mantissa is None:
            c.k_scale.copy_(torch.rand(H_kv, generator=g, device="cuda") + 1e-3)
        else:
            c.k_scale.copy_(torch.tensor(mantissa))
        c.v_scale.copy_(c.k_scale)
        pick = torch.randint(0, border.numel(), (n, H_kv, d), generator=g, device="cuda")
        x = (border[pick] * c.k_scale[:, None]).to(torch.bfloat16)
        x = torch.where(torch.rand(n, H_kv, d, generator=g, device="cuda") < 0.5, x, -x)
        binding.paged_append(c.handle(), None, x, x, c.table, c.kv_lens, cu_seqlens=_offsets([n]))
        want = (x.float() / c.k_scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        assert torch.equal(as_int(c.get(c.k, 0, 0, n)) & 0x7f, as_int(want) & 0x7f)
        assert torch.equal(c.get(c.v, 0, 0, n).float(), want.float())
