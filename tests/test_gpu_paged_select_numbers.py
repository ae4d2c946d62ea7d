"""Selection where a few pages' bounds, or a query, are no numbers: the choice is that of the definition in 64
bits, and the other pages cost what they cost without them."""

import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_paged_select import Boxes, _binding, _check  # noqa: E402

pytestmark = pytest.mark.gpu

INF, NAN = math.inf, math.nan


def _put(c, places, part, column, value):
    for i in places:
        c.bounds[c.ids[0][i], :, part, column] = value


def _mixed(c):         # NaN, both infinities, and a finite bound beside one
    n = len(c.ids[0])
    _put(c, (3, n // 2), 0, 5, NAN)
    _put(c, (4, n // 2 + 1), 1, 6, INF)
    _put(c, (n // 3,), 0, 7, -INF)
    _put(c, (n // 3 + 1, 9), 1, 8, -INF)
    _put(c, (12,), 1, slice(None), INF)


def _below(c):         # below every number for the heads with a positive element
    _put(c, range(2, len(c.ids[0]) - 2, 2), 1, 3, -INF)


def _many(c):          # more pages above all numbers than are chosen
    _put(c, range(1, len(c.ids[0]), 3), 1, 3, INF)


def _exactly(c):       # as many as are chosen, and one more below
    _put(c, range(40, 68), 1, 3, INF)
    _put(c, (20,), 1, 3, -INF)


def _large(c):         # products of the page's numbers that pass 32 bits beside an infinity, the other way
    _put(c, (17, 31), 1, 3, INF)
    _put(c, (17,), 0, slice(10, 20), 3e38)
    _put(c, (17,), 1, slice(20, 30), -3e38)


def _all_but_one(c):
    c.bounds[:, :, 1, 3] = INF
    c.bounds[c.ids[0][33]] = 1.0


def _zeros(c):         # the numbers are all 0
    c.bounds.zero_()
    _put(c, (50, 60), 1, 3, INF)
    _put(c, (4, 5, 6), 1, 3, -INF)


MAKES = [_mixed, _below, _many, _exactly, _large, _all_but_one, _zeros]


# (a cluster with all scores in one CTA, clusters whose CTAs decide together, four warps, one warp)
@pytest.mark.parametrize("make", MAKES)
@pytest.mark.parametrize("n,tokens,H_kv,d", [(700, 1, 1, 64), (3000, 1, 2, 128), (9000, 1, 1, 64), (700, 40, 8, 64), (90, 210, 8, 64)])
def test_pages_that_are_no_numbers(make, n, tokens, H_kv, d):
    c = Boxes([16 * n] + [16 * min(n, 90)] * (tokens - 1), H_kv, d, 16, make=make, seed=n)
    q = torch.randn(tokens, 3 * H_kv, d, device="cuda")
    for what in ("any", "positive", "one token negative"):
        if what != "any":
            q[..., 3] = q[..., 3].abs().clamp(min=0.1)
        if what == "one token negative":
            q[0, 0, 3] = -1.0
        _check(c, (q * (1e3 if make is _large else 1)).to(torch.bfloat16), None, 30, 1, 1, rows=[0, tokens - 1])


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("make", [None, _mixed, _zeros])
@pytest.mark.parametrize("n,tokens", [(700, 1), (9000, 1), (90, 1530)])
def test_queries_that_are_no_numbers(make, value, n, tokens):
    c = Boxes([16 * n] + [16 * min(n, 90)] * (tokens - 1), 1, 64, 16, make=make, seed=1)
    q = torch.randn(tokens, 3, 64, device="cuda").to(torch.bfloat16)
    q[0, 1, 5] = value
    _check(c, q, None, 30, 1, 1, rows=[0, tokens - 1])
    q[0] = 0
    _check(c, q, None, 30, 1, 1, rows=[0])
    q[0, 2, 63] = value
    _check(c, q, None, 30, 1, 1, rows=[0])


def _time(c, q):
    B = _binding()
    call = lambda: B.paged_select(c.handle, q, c.bounds, c.table, c.kv_lens, 64, keep_first=1, keep_last=2)  # noqa: E731
    for _ in range(3):
        call()
    best = math.inf
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(10):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("how", ["page", "query"])
def test_one_that_is_no_number_costs_little(how):
    """(With every page scored in 64 bits for the sake of one a call took 600 times as long.)"""
    c = Boxes([131072], 8, 128, 32)
    q = torch.randn(1, 32, 128, device="cuda", dtype=torch.bfloat16)
    plain = _time(c, q)
    if how == "page":
        c.bounds[c.ids[0][100], :, 0, 3] = NAN
    else:
        q[0, 5, 3] = NAN
    assert _time(c, q) < 20 * plain
