"""The paged key-value cache at the ends of its range."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from paged_common import E4M3_MAX, Cache, as_int, assert_attention, attention  # noqa: E402

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
