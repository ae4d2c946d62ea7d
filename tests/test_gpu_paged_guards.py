"""Offsets that are no offsets write nothing outside: every buffer of a call lies between margins that are
compared bit for bit, and so are the pages that no table names."""

import pytest

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from long_common import E8M0, Pages, as_int  # noqa: E402

pytestmark = pytest.mark.gpu

MARGIN = 16  # of each buffer's first dimension, on both sides
BAD = ([0, 90, 40, 120], [5, 60, 90, 120], [0, -7, 60, 500], [100, 50, 20, 10])


def _ints(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


class Guarded:
    """A buffer like `t` between margins of a pattern."""

    def __init__(self, t):
        shape = (t.shape[0] + 2 * MARGIN,) + tuple(t.shape[1:])
        self.all = torch.randint(0, 120, shape, device="cuda", dtype=torch.int32).to(_ints(t).dtype)
        self.n = t.shape[0]
        _ints(self.inside(t.dtype)).copy_(_ints(t))
        self.before = self.all.clone()

    def inside(self, dtype):
        return self.all.view(dtype)[MARGIN:MARGIN + self.n]

    def check(self, what, rows=None):
        """The margins, and the given rows, are as they were."""
        for part in (slice(0, MARGIN), slice(MARGIN + self.n, None)):
            assert torch.equal(self.all[part], self.before[part]), (what, part)
        if rows:
            at = torch.tensor(rows, device="cuda") + MARGIN
            assert torch.equal(self.all[at], self.before[at]), what


@pytest.mark.parametrize("tokens", [120, 24])  # (many and few tokens of a sequence)
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_bad_offsets_leave_other_memory_alone(bad, tokens):
    bad = [x if tokens == 120 else x // 5 for x in bad]
    c = Pages([200, 300, 100], 2, 64, 16, seed=3, spare=9)
    n_pages = c.k.shape[0]
    named = set(sum(c.ids, []))
    free = [p for p in range(n_pages) if p not in named]
    assert len(free) == 9
    g = {name: Guarded(getattr(c, name)) for name in ("k", "v", "k_exp", "v_exp")}
    g["bounds"] = Guarded(torch.zeros(n_pages, 2, 2, 64, device="cuda", dtype=torch.bfloat16))
    g["q_out"] = Guarded(torch.zeros(tokens, 4, 64, device="cuda", dtype=torch.bfloat16))
    g["pages"] = Guarded(torch.zeros(tokens, 2, 4, device="cuda", dtype=torch.int32))
    g["lens"] = Guarded(torch.zeros(tokens, device="cuda", dtype=torch.int32))
    fp8, bf16, i32 = c.k.dtype, torch.bfloat16, torch.int32
    cache = binding.PagedCache(g["k"].inside(fp8), g["v"].inside(fp8), k_scale=g["k_exp"].inside(E8M0),
                               v_scale=g["v_exp"].inside(E8M0))
    x = torch.randn(tokens, 2, 64, device="cuda", dtype=bf16)
    q = torch.randn(tokens, 4, 64, device="cuda", dtype=bf16)
    cu = torch.tensor(bad, dtype=i32, device="cuda")
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    binding.paged_append(cache, q, x, x, c.table, c.kv_lens, cu_seqlens=cu, inv_freq=freq, q_out=g["q_out"].inside(bf16))
    assert binding.attn_check(None) == 12
    binding.paged_bounds(cache, g["bounds"].inside(bf16), c.table, c.kv_lens, cu_seqlens=cu, tokens=tokens)
    assert binding.attn_check(None) == 12
    binding.paged_select(cache, q, g["bounds"].inside(bf16), c.table, c.kv_lens, 4, cu_seqlens=cu,
                         pages=g["pages"].inside(i32), lens=g["lens"].inside(i32))
    assert binding.attn_check(None) == 12
    for name in ("k", "v", "k_exp", "v_exp", "bounds"):
        g[name].check(name, free)
    for name in ("q_out", "pages", "lens"):
        g[name].check(name)


def test_the_check_sees_a_stray_write():
    g = Guarded(torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16))
    g.inside(torch.bfloat16)[1] = 1.0
    g.check("inside")
    with pytest.raises(AssertionError):
        g.check("row", [1])
    as_int(g.all.view(torch.bfloat16))[MARGIN + 4, 0] = 121
    with pytest.raises(AssertionError):
        g.check("margin")
