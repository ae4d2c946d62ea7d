"""The paged key-value cache at the ends of its range: quotients past 32 bits, rows of a
tile that belong to no token, query rows of zeros, waits that run out, small weights and
small steps over an e4m3 cache, chunks of very unequal lengths."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from paged_common import E4M3_MAX, Cache, as_int, assert_attention, attention  # noqa: E402
from paged_weights import SMALL, bound, small_weights  # noqa: E402

WIDE = 100000  # tokens that a page table can hold: a chunk call then takes the tensor-core kernel


@pytest.fixture(autouse=True)
def _clean():
    assert binding.attn_check(None) == 0
    yield
    assert binding.attn_check(None) == 0


def _q(n, H, d, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, H, d, generator=g, device="cuda").to(torch.bfloat16)


def _offsets(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


def _table(c, tokens):
    """The page table, or one that could hold that many tokens a sequence."""
    table = torch.full((len(c.lens), max(c.width, tokens // c.page)), -7, dtype=torch.int32, device="cuda")
    table[:, :c.width] = c.table
    return table


def _want(c, q, new, scale, causal=True):
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


@pytest.mark.parametrize("x, scale", [(3e38, 0.5), (3.3e38, 0.9375), (1e37, 0.01), (1e30, 1e-9), (1e20, 1e-20), (1e10, 1e-29),
                                      (1e9, 1e-29), (448.0, 0.9), (3e38, 2e-30)])
def test_append_finite_values_past_the_range(x, scale):
    """A finite value whose quotient by the scale passes 448 is stored as 448 of its sign,
    the same where that quotient, or the product with the rounded inverse, passes 32 bits."""
    c = Cache([2], 2, 64, 16, "e4m3")
    c.k_scale.fill_(scale)
    c.v_scale.fill_(scale)
    k = torch.full((2, 2, 64), x, device="cuda")
    k[:, :, ::2] *= -1
    k[1, 1, :] = 0
    k = k.to(torch.bfloat16)
    assert bool(torch.isfinite(k).all())
    binding.paged_append(c.handle(), None, k, k, c.table, c.kv_lens, cu_seqlens=_offsets([2]))
    want = torch.where(k == 0, torch.zeros_like(k), torch.copysign(torch.full_like(k, E4M3_MAX), k)).float()
    for cache in (c.k, c.v):
        assert torch.equal(c.get(cache, 0, 0, 2).float(), want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_rows_of_zeros_and_tiny_rows_over_e4m3(d, wide, causal):
    """Rows of zeros and of tiny values between rows of large ones, whose scale is small: the
    product of the scales and a row's power of two passes below 32 bits in some rows of a
    warp and not in others."""
    new = [150, 200]
    c = Cache([300, 200], 2, d, 16, "e4m3")
    q = _q(350, 8, d).float() * 2.0 ** 40
    q[::3] = 0.0
    q[1::5] *= 2.0 ** -150
    q[7, :4] = 0.0
    q = q.to(torch.bfloat16)
    for scale in (2.0 ** -40 / math.sqrt(d), -(2.0 ** -40) / math.sqrt(d), 1e-36):
        o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new), scale=scale, causal=causal)
        assert_attention(o, lse, *_want(c, q, new, scale, causal), what=scale)


def _fill_query_tiles(d, kind, factor):
    """A chunk call that fills every row of the query tiles of all CTAs."""
    c = Cache([10300], 4, d, 64, kind, seed=5)
    q = (_q(10300, 4, d, seed=6).float() * factor).to(torch.bfloat16)
    binding.paged_forward(c.handle(), q, c.table, c.kv_lens, _offsets([10300]))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 7, 24])
def test_chunk_does_not_depend_on_the_call_before(group, d, kind):
    """Groups that do not divide a tile's 128 rows leave rows that no copy writes: what an
    earlier call left there changes no bit of a result."""
    new = [200, 50]
    c = Cache([2000, 1500], 2, d, 64, kind, seed=2)
    h, q, table, cu = c.handle(), _q(250, 2 * group, d), _table(c, WIDE), _offsets(new)
    got = []
    for factor in (0.0, 40.0, 0.01, -40.0):
        _fill_query_tiles(d, kind, factor)
        got.append(binding.paged_forward(h, q, table, c.kv_lens, cu))
    assert_attention(*got[0], *_want(c, q, new, 1.0 / math.sqrt(d)))
    for o, lse in got[1:]:
        assert torch.equal(as_int(o), as_int(got[0][0])) and torch.equal(lse, got[0][1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_chunk_does_not_depend_on_rows_of_others(group, kind):
    """The rows of q behind the last sequence, and the next sequence's, lie in the last
    tile of one: they change no bit of it."""
    d, new = 128, [190, 30]
    c = Cache([2000, 1500], 2, d, 64, kind, seed=3)
    h, table, cu = c.handle(), _table(c, WIDE), _offsets(new)
    q = _q(300, 2 * group, d)
    got = []
    for factor in (1.0, 40.0):
        x = q.clone()
        x[220:] *= factor
        got.append([t for t in binding.paged_forward(h, x, table, c.kv_lens, cu)])
    assert torch.equal(as_int(got[0][0][:220]), as_int(got[1][0][:220]))
    assert torch.equal(got[0][1][:, :220], got[1][1][:, :220])
    x = q.clone()
    x[190:220] *= 40.0
    o, lse = binding.paged_forward(h, x, table, c.kv_lens, cu)
    assert torch.equal(as_int(o[:190]), as_int(got[0][0][:190])) and torch.equal(lse[:, :190], got[0][1][:, :190])


SHORT_LIMIT = 2_000_000  # cycles, about a millisecond


def _with_a_warp_that_leaves(call):
    """The call's status when one warp of each CTA leaves as if its wait had run out, and the
    outputs of the same call before and after it."""
    before = [t.clone() for t in call()]
    assert binding.attn_check(None) == 0
    old = binding.attn_set_wait_limit(SHORT_LIMIT)
    try:
        assert binding.attn_debug_inject(binding.FAULT_LEAVE_WARP) == 0
        call()
        status = binding.attn_check(None)
    finally:
        assert binding.attn_debug_inject(binding.FAULT_NONE) == 0
        binding.attn_set_wait_limit(old)
    after = call()
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    return status


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [0, WIDE])
def test_a_warp_that_leaves_ends_one_token_attention(wide, kind):
    """The other warps give up where they wait for it: the call ends, reports the time-out,
    and the next one is right."""
    c = Cache([2000, 700], 2, 128, 16, kind)
    h, q, table = c.handle(), _q(2, 8, 128), _table(c, wide)
    assert _with_a_warp_that_leaves(lambda: binding.paged_decode(h, q, table, c.kv_lens)) == 9  # ATTN_ERR_TIMEOUT


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [[300, 200], [1024]])
def test_a_warp_that_leaves_ends_chunk_attention(new, d, kind):
    """The same in the tensor-core kernel, where a warp leaves before the tile's epilogue."""
    c = Cache([n + 900 for n in new], 2, d, 16, kind)
    h, q, table, cu = c.handle(), _q(sum(new), 8, d), _table(c, WIDE), _offsets(new)
    assert _with_a_warp_that_leaves(lambda: binding.paged_forward(h, q, table, c.kv_lens, cu)) == 9


def _lost(q, k, v, scale, last):
    """Of q [n, H_q, d] over k, v [L, H_kv, d]: the sum of |v_j| over the keys whose weight
    is below 2^-21 of the row's largest, by the sum of weights [n, H_q, d]."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1).transpose(0, 1), v.repeat_interleave(g, 1).transpose(0, 1)
    s = q.double().transpose(0, 1) @ k.transpose(1, 2) * scale
    s = s.masked_fill(torch.arange(k.shape[1], device=q.device)[None] >= last[:, None], -math.inf)
    w = torch.exp(s - s.amax(-1, keepdim=True))
    small = (w < 2.0 ** -21) & (s > -math.inf)
    return ((small.double() @ v.abs()) / w.sum(-1, keepdim=True)).transpose(0, 1)


def _assert_e4m3(o, c, q, new, scale, causal):
    want, size, _ = _want(c, q, new, scale, causal)
    lost, t0 = [], 0
    for b, n in enumerate(new):
        L = c.lens[b]
        last = torch.full((n,), L, device="cuda")
        if causal:
            last = L - n + 1 + torch.arange(n, device="cuda")
        lost.append(_lost(q[t0:t0 + n], c.keys[b], c.values[b], scale, last))
        t0 += n
    err, most = (o.double() - want).abs(), bound(want, size, torch.cat(lost))
    assert bool((err <= most).all()), float((err / most).max())


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", SMALL)
def test_small_weights_keep_eleven_bits_over_e4m3(exponent, d, n, wide):
    """Weights that bf16, or fp16 without the factor of 2^7, would round past the bound (as
    the planted mistakes show on the CPU), next to weights of 1."""
    c = Cache([200], 1, d, 16, "e4m3")
    c.k_scale.fill_(0.25)
    c.v_scale.fill_(0.5)
    w, v = small_weights(exponent, d)
    k = torch.zeros(200, 1, d, device="cuda")
    k[::16, 0, 0] = 4.0
    v = v.cuda()[:, None] / 0.5
    for cache, x in ((c.k, k), (c.v, v)):
        c.put(cache, 0, 0, x.to(torch.float8_e4m3fn))
    c.keys, c.values = [k.double() * 0.25], [v * 0.5]
    q = torch.zeros(n, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    scale = float(torch.tensor(exponent * math.log(2.0)))
    if n == 1:
        o, _ = binding.paged_decode(c.handle(), q, _table(c, wide), c.kv_lens, scale=scale)
    else:
        o, _ = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets([n]), scale=scale, causal=False)
    _assert_e4m3(o, c, q, [n], scale, False)


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("new, lens, H_q, H_kv, d, page", [
    ([1, 1, 1], [1, 700, 3000], 8, 2, 128, 16), ([1], [9000], 5, 1, 64, 32), ([4, 2], [500, 64], 16, 4, 128, 64),
    ([300, 40], [300, 900], 8, 2, 128, 16), ([129, 65], [2000, 65], 10, 2, 64, 32)])
def test_attention_over_e4m3_keeps_fp16_weights(new, lens, H_q, H_kv, d, page, wide):
    """Random sequences within the bound of fp16 weights, not bf16's."""
    c = Cache(lens, H_kv, d, page, "e4m3", seed=7)
    q, scale = _q(sum(new), H_q, d), 1.0 / math.sqrt(d)
    if max(new) == 1:
        o, _ = binding.paged_decode(c.handle(), q, _table(c, wide), c.kv_lens)
    else:
        o, _ = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new))
    _assert_e4m3(o, c, q, new, scale, max(new) > 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("wide", [0, 3000, WIDE])
def test_one_prompt_among_many_single_tokens(wide, kind):
    """The host knows the mean of the chunks only: a prompt of 700 tokens, in the middle of 255
    sequences of one token each, and one without any."""
    new = [1] * 100 + [700, 0] + [1] * 155
    lens = [17 + 3 * i for i in range(100)] + [900, 40] + [5 + 2 * i for i in range(155)]
    c = Cache(lens, 2, 64, 16, kind, seed=8)
    q = _q(sum(new), 8, 64)
    o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, _offsets(new))
    assert_attention(o, lse, *_want(c, q, new, 1.0 / 8.0))
