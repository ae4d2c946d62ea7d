"""A paged cache with a power of two for each page and KV head: appending to it and
attention over it, against definitions in 64 bits (bounds in paged_common)."""

import math

import pytest
import torch

from paged_common import BF16, E4M3, E4M3_MAX, as_int, assert_attention, attention, turned
from long_common import Pages, encoded, exponent, values_of

pytestmark = pytest.mark.gpu


def _binding():
    from exact_attention_15_gb300 import binding
    return binding


def _ok():
    assert _binding().attn_check(None) == 0


def _inv_freq(rotary, base=10000.0):
    return base ** (-torch.arange(rotary // 2, dtype=torch.float64, device="cuda") * 2 / rotary)


def _cu(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- attention

EXPS = {
    "near": ((-8, -4), (-8, -4)),
    "far": ((-12, -3), (-46, 24)),   # the values' sizes differ by 2^70
    "tiny": ((-50, -40), (-64, -60)),
}


@pytest.mark.parametrize("exps", EXPS)
@pytest.mark.parametrize("lens,H_kv,group,d,page", [
    ([1], 1, 1, 64, 16), ([777], 8, 4, 128, 16), ([0, 1, 63, 64, 65, 200], 2, 5, 64, 32),
    ([300, 17, 4096, 900], 4, 8, 128, 64), ([31, 500], 3, 12, 64, 256), ([2000] * 3, 2, 16, 128, 128)])
def test_decode(lens, H_kv, group, d, page, exps):
    c = Pages(lens, H_kv, d, page, *EXPS[exps], seed=len(lens))
    q = torch.randn(len(lens), H_kv * group, d, device="cuda", dtype=torch.bfloat16)
    o, lse = _binding().paged_decode(c.handle(), q, c.table, c.kv_lens)
    for b, n in enumerate(lens):
        want, want_abs, want_lse = c.attention(q[b:b + 1], b, 1 / math.sqrt(d), torch.tensor([n], device="cuda"))
        assert_attention(o[b:b + 1], lse[b][:, None], want, want_abs, want_lse, (b, n))
    _ok()


# many keys in all: the units are dealt out over the GPU and joined
@pytest.mark.parametrize("d,page,group", [(128, 64, 4), (64, 16, 16), (128, 16, 1)])
def test_decode_dealt_out(d, page, group):
    lens = [9000, 1, 20000, 333]
    c = Pages(lens, 2, d, page, (-9, -5), (-20, 6), seed=7)
    q = torch.randn(4, 2 * group, d, device="cuda", dtype=torch.bfloat16)
    o, lse = _binding().paged_decode(c.handle(), q, c.table, c.kv_lens)
    for b, n in enumerate(lens):
        want, want_abs, want_lse = c.attention(q[b:b + 1], b, 1 / math.sqrt(d), torch.tensor([n], device="cuda"))
        assert_attention(o[b:b + 1], lse[b][:, None], want, want_abs, want_lse, (b, n))
    again = _binding().paged_decode(c.handle(), q, c.table, c.kv_lens)
    assert torch.equal(as_int(again[0]), as_int(o)) and torch.equal(again[1], lse)
    _ok()


CHUNKS = [
    ([1], [0], 1, 1, 64, 16), ([4, 3, 1], [700, 0, 90], 2, 4, 128, 32), ([130], [0], 2, 4, 128, 64),
    ([300, 5, 257], [100, 0, 1000], 2, 4, 64, 16), ([700], [1500], 4, 8, 128, 16), ([513, 1], [0, 40], 1, 1, 64, 256),
    ([2000, 100], [0, 3000], 4, 8, 128, 128), ([600, 600, 600, 600], [0, 10, 500, 64], 8, 4, 64, 32)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("exps", ["near", "far"])
@pytest.mark.parametrize("new,ctx,H_kv,group,d,page", CHUNKS)
def test_chunks(new, ctx, H_kv, group, d, page, exps, causal):
    lens = [n + x for n, x in zip(new, ctx)]
    c = Pages(lens, H_kv, d, page, *EXPS[exps], seed=sum(new))
    T = sum(new)
    q = torch.randn(T + 2, H_kv * group, d, device="cuda", dtype=torch.bfloat16)  # two rows behind the last
    out, lse = torch.full_like(q, 7.0), torch.full((H_kv * group, T + 2), 7.0, device="cuda")
    _binding().paged_forward(c.handle(), q, c.table, c.kv_lens, _cu(new), causal=causal, out=out, lse=lse)
    t0 = 0
    for b, n in enumerate(new):
        last = torch.full((n,), lens[b], device="cuda")
        if causal:
            last = last - n + 1 + torch.arange(n, device="cuda")
        want, want_abs, want_lse = c.attention(q[t0:t0 + n], b, 1 / math.sqrt(d), last)
        assert_attention(out[t0:t0 + n], lse[:, t0:t0 + n], want, want_abs, want_lse, b)
        t0 += n
    assert bool((out[T:] == 7).all()) and bool((lse[:, T:] == 7).all())
    _ok()


@pytest.mark.parametrize("new", [None, 300])
def test_negative_and_zero_scale(new):
    """Any finite scale: the scores' order turns round, or all weights are equal."""
    c = Pages([400], 2, 64, 32, (-8, -4), (-9, -2), seed=3)
    n = new or 1
    q = torch.randn(n, 4, 64, device="cuda", dtype=torch.bfloat16)
    for scale in (-0.1, 0.0):
        if new:
            o, lse = _binding().paged_forward(c.handle(), q, c.table, c.kv_lens, _cu([n]), scale=scale, causal=False)
        else:
            o, lse = _binding().paged_decode(c.handle(), q, c.table, c.kv_lens, scale=scale)
            lse = lse.t()
        want, want_abs, want_lse = attention(q, c.sequence("k", 0), c.sequence("v", 0), scale,
                                             torch.full((n,), 400, device="cuda"))
        assert_attention(o, lse, want, want_abs, want_lse, scale)
    _ok()


@pytest.mark.parametrize("new", [None, 200])
def test_exponents_outside_the_range_count_as_its_ends(new):
    c = Pages([200], 1, 64, 16, seed=4)
    c.k_exp.fill_(127 - 6)
    c.v_exp.fill_(0)
    c.v_exp[c.ids[0][3]] = 10   # both count as 2^-64
    q = torch.randn(new or 1, 2, 64, device="cuda", dtype=torch.bfloat16)
    call = (lambda: _binding().paged_forward(c.handle(), q, c.table, c.kv_lens, _cu([new]))[0]) if new else (
        lambda: _binding().paged_decode(c.handle(), q, c.table, c.kv_lens)[0])
    o = call()
    c.v_exp.fill_(127 - 64)
    assert torch.equal(as_int(call()), as_int(o))
    c.v_exp.fill_(255)
    o = call()
    c.v_exp.fill_(127 + 24)
    assert torch.equal(as_int(call()), as_int(o))
    _ok()


def test_pages_of_zeros():
    """Zero values with the smallest exponent beside others: their weights still count in the sum."""
    c = Pages([256], 1, 64, 64, (-6, -6), (-6, -6), seed=5)
    for i in (0, 2):
        as_int(c.v)[c.ids[0][i]] = 0
        c.v_exp[c.ids[0][i]] = 127 - 64
    for n in (1, 256):
        q = torch.randn(n, 4, 64, device="cuda", dtype=torch.bfloat16)
        o, lse = _binding().paged_forward(c.handle(), q, c.table, c.kv_lens, _cu([n]), causal=False)
        want, want_abs, want_lse = attention(q, c.sequence("k", 0), c.sequence("v", 0), 0.125, torch.full((n,), 256, device="cuda"))
        assert_attention(o, lse, want, want_abs, want_lse, n)
    _ok()


@pytest.mark.parametrize("n", [1, 200])
def test_weights_across_the_whole_range(n):
    """Equal keys, so equal weights: pages of the smallest and of the largest scale share the sum,
    and with -inf-like scores on the large ones the small ones' values come out."""
    c = Pages([512], 1, 64, 64, (-6, -6), (-64, -64), seed=8)
    for i in (1, 4):
        c.v_exp[c.ids[0][i]] = 127 + 24
    as_int(c.k)[:] = as_int(c.k)[c.ids[0][0], :, :1]
    q = torch.randn(n, 2, 64, device="cuda", dtype=torch.bfloat16)
    call = lambda: _binding().paged_forward(c.handle(), q, c.table, c.kv_lens, _cu([n]), causal=False)  # noqa: E731
    o, lse = call()
    want, want_abs, want_lse = attention(q, c.sequence("k", 0), c.sequence("v", 0), 0.125, torch.full((n,), 512, device="cuda"))
    assert_attention(o, lse, want, want_abs, want_lse, n)
    # scores 256 below: weights of 0
    q = torch.full_like(q, 4.0)
    as_int(c.k)[:] = as_int(torch.ones(1, device="cuda").to(c.k.dtype))
    for i in (1, 4):
        as_int(c.k)[c.ids[0][i]] = as_int(torch.full((1,), -64.0, device="cuda").to(c.k.dtype))
    c.k_exp.fill_(127)
    o, lse = call()
    want, want_abs, want_lse = attention(q, c.sequence("k", 0), c.sequence("v", 0), 0.125, torch.full((n,), 512, device="cuda"))
    assert_attention(o, lse, want, want_abs, want_lse, n)
    _ok()


# ---------------------------------------------------------------- appending

def _append(c, new, H_q, rotary, interleaved, x=None, fused=True, seed=1):
    """Appends to c (whose lengths count the new tokens), checks everything against the
    definition, and returns what was appended."""
    B = _binding()
    H_kv, d, page = c.H_kv, c.d, c.page
    T = sum(new)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if x is None:
        x = torch.randn(T, H_q + 2 * H_kv, d, generator=g, device="cuda", dtype=torch.bfloat16)
    if not fused:
        x = x.clone()
    q, k, v = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    freq = _inv_freq(rotary) if rotary else None
    before = {n: getattr(c, n).clone() for n in ("k", "v", "k_exp", "v_exp")}
    want = {n: t.clone() for n, t in before.items()}
    free = {n: torch.zeros(c.k.shape, dtype=torch.float64, device="cuda") for n in ("k", "v")}  # allowed deviation
    cu = None if all(n == 1 for n in new) else _cu(new)
    got = B.paged_append(c.handle(), q if H_q else None, k, v, c.table, c.kv_lens, cu_seqlens=cu, inv_freq=freq,
                         interleaved=interleaved)
    _ok()
    t0 = 0
    for b, n in enumerate(new):
        begin = c.lens[b] - n
        pos = torch.arange(begin, c.lens[b], device="cuda")
        for name, new_x in (("k", k), ("v", v)):
            raw = new_x[t0:t0 + n].double()
            if name == "k" and rotary:
                y, pair = turned(new_x[t0:t0 + n].cpu(), pos.cpu(), freq.cpu(), interleaved)
                y, pair = y.cuda(), pair.cuda()
            else:
                y, pair = raw, torch.zeros_like(raw)
            for i in range(begin // page, (c.lens[b] - 1) // page + 1) if n else []:
                p, r0 = c.ids[b][i], max(0, begin - i * page)
                lo, hi = max(0, i * page - begin), min(n, (i + 1) * page - begin)
                for h in range(H_kv):
                    size = raw[lo:hi, h].abs()
                    most = float(size[size < math.inf].max()) if bool((size < math.inf).any()) else 0.0
                    e = exponent(most * (1.5 if name == "k" and rotary else 1.0))
                    if r0:
                        old = max(-64, min(24, int(before[name + "_exp"][p, h]) - 127))
                        e = max(e, old)
                        if e > old:
                            kept = encoded(before[name][p, h, :r0].double(), e - old)
                            want[name][p, h, :r0] = kept
                        if e == old:
                            want[name + "_exp"][p, h] = before[name + "_exp"][p, h]
                    if not r0 or e > old:
                        want[name + "_exp"][p, h] = e + 127
                    want[name][p, h, r0:r0 + hi - lo] = encoded(y[lo:hi, h], e)
                    # half a step of e4m3 relative to the value (its smallest normal number
                    # at least), and the 32-bit turn's error, both in stored units
                    size = torch.ldexp(y[lo:hi, h].abs(), torch.full((1,), float(-e), dtype=torch.float64, device="cuda"))
                    turn = torch.ldexp(pair[lo:hi, h], torch.full((1,), float(-e), dtype=torch.float64, device="cuda"))
                    free[name][p, h, r0:r0 + hi - lo] = torch.where(
                        turn > 0, 2 * E4M3 * size.clamp(2.0 ** -6, E4M3_MAX) + 2.0 ** -20 * turn, 0.0)
        t0 += n
    for name in ("k", "v"):
        assert torch.equal(getattr(c, name + "_exp"), want[name + "_exp"]), name
        # equal bits but where a turned value lies next to a border: there one step at most
        a, w = getattr(c, name), want[name]
        differ = as_int(a) != as_int(w)
        err = (a.double() - w.double()).abs()
        assert bool((~differ | (err <= free[name])).all()), (name, int(differ.sum()))
        assert float(differ.sum()) <= 1e-3 * max(1, T * H_kv * d) + 4, name
    return x, got


@pytest.mark.parametrize("H_q,H_kv,d,page,rotary,interleaved", [
    (8, 2, 128, 16, 128, False), (6, 3, 64, 32, 32, True), (4, 4, 64, 16, 0, False), (0, 1, 128, 256, 64, False),
    (16, 1, 128, 64, 128, True), (32, 8, 128, 128, 64, False), (20, 10, 128, 64, 48, False), (3, 3, 64, 256, 16, True),
    (34, 17, 64, 32, 64, False)])
@pytest.mark.parametrize("new,ctx", [
    ([1], [0]), ([1, 1, 1, 1, 1], [0, 15, 16, 17, 300]), ([5, 1, 40, 0, 33], [0, 31, 100, 9, 7]), ([700, 129], [0, 63]),
    ([300], [1])])
def test_append(new, ctx, H_q, H_kv, d, page, rotary, interleaved):
    lens = [n + x for n, x in zip(new, ctx)]
    # pages of smaller values than the new ones (they grow) and of larger ones (they stay)
    c = Pages(lens, H_kv, d, page, (-9, -3), (-9, -3), seed=sum(lens))
    x, q = _append(c, new, H_q, rotary, interleaved, fused=bool(sum(new) & 1))
    if not H_q:
        return
    freq = _inv_freq(rotary) if rotary else None
    pos = torch.tensor([ctx[b] + i for b, n in enumerate(new) for i in range(n)])
    y, pair = turned(x[:, :H_q].cpu(), pos, None if freq is None else freq.cpu(), interleaved)
    err = (q.cpu().double() - y).abs()
    assert bool((err <= (BF16 * y.abs() + 2.0 ** -20 * pair if rotary else 0 * err)).all())


@pytest.mark.parametrize("middle,page", [(40, 16), (80, 16), (80, 64)])  # (few and many tokens of a sequence)
def test_append_values_of_every_size(middle, page):
    """Zeros, the smallest and largest numbers, infinities and NaN among the new values."""
    c = Pages([5, middle, 1], 2, 64, page, seed=9)
    x = torch.randn(6 + middle, 4, 64, device="cuda", dtype=torch.bfloat16)
    x[0] = 0                       # first token of a sequence: zeros
    x[5:12] *= 2.0 ** -100         # a page of numbers below 2^-64: the exponent's lower end
    x[5:21, 2] = 2.0 ** -90
    x[21:37, 1] = 3e38             # above 448 2^24
    x[22:30, 3, 5] = math.inf
    x[23, 2, 7], x[24, 2, 8] = math.nan, -math.inf
    x[-1, 0] = 448.0 * 2.0 ** -5   # the border of an exponent, and one step above it
    x[-1, 1] = 450.0 * 2.0 ** -5
    B = _binding()
    B.paged_append(c.handle(), None, x[:, :2].contiguous(), x[:, 2:].contiguous(), c.table, c.kv_lens, cu_seqlens=_cu([5, middle, 1]))
    _ok()
    t0 = 0
    for b, n in enumerate(c.lens):
        for i in range(-(-n // page)):
            p, rows = c.ids[b][i], slice(t0 + page * i, t0 + min(n, page * i + page))
            for h in range(4):
                name, hh = ("k", h) if h < 2 else ("v", h - 2)
                y = x[rows, h].double()
                size = y.abs()
                e = exponent(float(torch.where(size < math.inf, size, torch.zeros_like(size)).max()))
                assert int(getattr(c, name + "_exp")[p, hh]) == e + 127, (b, i, h)
                stored = getattr(c, name)[p, hh, :y.shape[0]]
                want = encoded(torch.where(y.isnan(), torch.zeros_like(y), y), e)
                assert torch.equal(as_int(torch.where(y.isnan(), torch.zeros_like(stored.float()), stored.float()).to(stored.dtype)),
                                   as_int(want)), (b, i, h)
                assert torch.equal(stored.float().isnan(), y.isnan())
        t0 += n


def test_append_token_by_token_grows_pages():
    """Growing values, one token at a time: each page's exponent follows, and its rows keep their
    values to half a step of the last encoding each time."""
    n, page, d = 40, 16, 128
    c = Pages([n], 1, d, page, seed=2)
    c.k_exp.fill_(200), c.v_exp.fill_(3)  # left by an earlier owner: not read for a fresh page
    x = torch.randn(n, 2, d, device="cuda", dtype=torch.bfloat16) * (1.2 ** torch.arange(n, device="cuda"))[:, None, None]
    x = x.to(torch.bfloat16)
    for i in range(n):
        c.kv_lens.fill_(i + 1)
        _binding().paged_append(c.handle(), None, x[i:i + 1, :1].contiguous(), x[i:i + 1, 1:].contiguous(), c.table, c.kv_lens)
    _ok()
    c.lens = [n]
    for name, col in (("k", 0), ("v", 1)):
        for i in range(-(-n // page)):
            rows = x[i * page:(i + 1) * page, col].double()
            e = exponent(float(rows.abs().max()))
            p = c.ids[0][i]
            assert int(getattr(c, name + "_exp")[p, 0]) == e + 127
            got = values_of(getattr(c, name)[p], getattr(c, name + "_exp")[p])[0, :rows.shape[0]]
            # 16 encodings at most: each normal value rounds once (the steps of finer scales are
            # those of coarser ones), below 2^-6 of the stored range half of 2^-9 a time
            assert bool(((got - rows).abs() <= E4M3 * rows.abs() + 16 * 2.0 ** (e - 10)).all())


def test_append_bad_pages_and_lengths():
    """Page indices and lengths outside the cache write nothing and are recorded."""
    B = _binding()
    for bad, n in ((-1, 10), (10 ** 6, 10), (-1, 40), (10 ** 6, 40)):
        c = Pages([n + 10, n + 10], 2, 64, 16, seed=1)
        c.table[0, 1] = bad
        before = {m: getattr(c, m).clone() for m in ("k", "v", "k_exp", "v_exp")}
        x = torch.randn(2 * n, 2, 64, device="cuda", dtype=torch.bfloat16)
        B.paged_append(c.handle(), None, x, x, c.table, c.kv_lens, cu_seqlens=_cu([n, n]))
        assert B.attn_check(None) == 13
        ids = set(c.ids[0][:1] + c.ids[0][2:] + c.ids[1])
        for p in range(c.k.shape[0]):
            if p not in ids:
                for m, t in before.items():
                    assert torch.equal(as_int(getattr(c, m)[p]), as_int(t[p])), (m, p)
    c = Pages([20], 1, 64, 16, seed=1, width=2)
    before = c.k.clone()
    x = torch.randn(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    c.kv_lens.fill_(-5)
    B.paged_append(c.handle(), None, x, x, c.table, c.kv_lens, cu_seqlens=_cu([4]))
    assert B.attn_check(None) == 13
    assert torch.equal(as_int(c.k), as_int(before))


@pytest.mark.parametrize("n", [8, 50])  # (few and many tokens of a sequence)
def test_append_padding_rows(n):
    """A sequence that is shorter than its rows: only the rows at positions from 0 on."""
    c = Pages([3, n + 12], 1, 64, 16, seed=6)
    x = torch.randn(n + 9, 4, 64, device="cuda", dtype=torch.bfloat16)
    q_out = torch.full((n + 9, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    freq = _inv_freq(64)
    _binding().paged_append(c.handle(), x[:, :2], x[:, 2:3], x[:, 3:], c.table, c.kv_lens, cu_seqlens=_cu([8, n]), inv_freq=freq,
                            q_out=q_out)
    _ok()
    assert bool((q_out[:5] == 7).all()) and bool((q_out[8 + n:] == 7).all())
    assert not bool((q_out[5:8 + n] == 7).all(dim=2).any())
    e = exponent(float(x[5:8, 3].abs().max()))
    assert int(c.v_exp[c.ids[0][0], 0]) == e + 127
    assert torch.equal(as_int(c.v[c.ids[0][0], 0, :3]), as_int(encoded(x[5:8, 3].double(), e)))
    assert bool((as_int(c.v[c.ids[0][0], 0, 3:]) == 0x7F).all())
