"""How many bits the weights have over pages with scales, by the kernel that a call takes, and what
pages of far larger values than others do to the outputs (bounds in paged_common and paged_weights)."""

import math

import pytest

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from long_common import Pages, as_int  # noqa: E402
from paged_common import assert_attention, attention  # noqa: E402
from paged_weights import SMALL, bound, small_weights  # noqa: E402

pytestmark = pytest.mark.gpu

WIDE = 400000  # tokens that a page table can hold: a chunk call then takes the tensor-core kernel
STREAM, CHUNK = "paged_stream_kernel", "paged_fwd_kernel"


def _table(c, tokens):
    """The page table, or one that could hold that many tokens a sequence."""
    table = torch.full((len(c.lens), max(c.width, tokens // c.page)), -7, dtype=torch.int32, device="cuda")
    table[:, :c.width] = c.table
    return table


def _attend(c, q, wide, scale):
    """Outputs and log-sum-exps of q's rows over all keys of c's one sequence, and the kernel that ran."""
    n = q.shape[0]
    binding.attn_profile_read()
    binding.attn_profile_enable(True)
    try:
        if n == 1:
            o, lse = binding.paged_decode(c.handle(), q, _table(c, wide), c.kv_lens, scale=scale)
            lse = lse.t()
        else:
            cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
            o, lse = binding.paged_forward(c.handle(), q, _table(c, wide), c.kv_lens, cu, scale=scale, causal=False)
        ran = [k for k, _ in binding.attn_profile_read() if k in (STREAM, CHUNK)]
    finally:
        binding.attn_profile_enable(False)
    assert binding.attn_check(None) == 0
    assert len(ran) == 1
    return o, lse, ran[0]


@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", SMALL)
def test_small_weights(exponent, d, n, wide):
    """Weights that bf16, or fp16 without the factor of 2^7, would round past the bound of eleven bits,
    next to weights of 1: the kernel for few tokens holds them, that for chunks holds eight bits."""
    c = Pages([200], 1, d, 16, (-2, -2), (-1, -1))
    w, v = small_weights(exponent, d)
    k = torch.zeros(200, 1, d, device="cuda")
    k[::16, 0, 0] = 4.0
    v = v.cuda()[:, None] / 0.5
    for name, x in (("k", k), ("v", v)):
        for i, p in enumerate(c.ids[0]):
            rows = x[16 * i:16 * i + 16].to(torch.float8_e4m3fn)
            as_int(getattr(c, name))[p, 0, :rows.shape[0]] = as_int(rows[:, 0].contiguous())
    assert torch.equal(c.sequence("k", 0), k.double() * 0.25) and torch.equal(c.sequence("v", 0), v * 0.5)
    q = torch.zeros(n, 2, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    scale = float(torch.tensor(exponent * math.log(2.0)))
    o, lse, ran = _attend(c, q, wide, scale)
    assert ran == (CHUNK if n == 130 and wide else STREAM)
    want, want_abs, want_lse = attention(q, c.sequence("k", 0), c.sequence("v", 0), scale, torch.full((n,), 200, device="cuda"))
    assert_attention(o, lse, want, want_abs, want_lse)
    if ran == STREAM:
        err = (o.double() - want).abs()
        assert bool((err <= bound(want, want_abs, torch.zeros_like(want))).all()), float((err / want_abs).max())


FAR = [([2000, 100], [0, 3000], 4, 8, 128, 128), ([600, 600, 600, 600], [0, 10, 500, 64], 8, 4, 64, 32),
       ([700], [1500], 4, 8, 128, 16), ([300], [1500], 2, 4, 64, 64)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx,H_kv,group,d,page", FAR)
def test_chunks_over_far_scales_lose_nothing(new, ctx, H_kv, group, d, page, causal):
    """The kernel for chunks widens the values with their scales, so its weights are relative to nothing but
    themselves: the bound of a bf16 cache, without the kernel for few tokens' absolute part."""
    lens = [n + x for n, x in zip(new, ctx)]
    c = Pages(lens, H_kv, d, page, (-12, -3), (-46, 24), seed=sum(new) + causal)
    q = torch.randn(sum(new), H_kv * group, d, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    binding.attn_profile_read()
    binding.attn_profile_enable(True)
    try:
        out, lse = binding.paged_forward(c.handle(), q, _table(c, WIDE), c.kv_lens, cu, causal=causal)
        assert CHUNK in [k for k, _ in binding.attn_profile_read()]
    finally:
        binding.attn_profile_enable(False)
    assert binding.attn_check(None) == 0
    t0 = 0
    for b, n in enumerate(new):
        last = torch.full((n,), lens[b], device="cuda")
        if causal:
            last = last - n + 1 + torch.arange(n, device="cuda")
        want, want_abs, want_lse = attention(q[t0:t0 + n], c.sequence("k", b), c.sequence("v", b), 1 / math.sqrt(d), last)
        assert_attention(out[t0:t0 + n], lse[:, t0:t0 + n], want, want_abs, want_lse, b)
        t0 += n


@pytest.mark.parametrize("n", [1, 130])
@pytest.mark.parametrize("up", [8, 18, 24, 30])
def test_an_outlier_channel_in_one_page(up, n):
    """One page of four holds 448 2^(up - 6) in one channel and zeros elsewhere, the others values up to
    448 2^-6. The kernel for few tokens keeps eleven bits of every weight of a stored value from 2^-21 of the
    largest on, and the others to 2^-32 of it; the kernel for chunks loses nothing in the other channels."""
    d = 64
    c = Pages([256], 1, d, 64, (-8, -4), (-6, -6), seed=up)
    page = c.ids[0][1]
    c.v_exp[page] = 127 - 6 + up
    as_int(c.v)[page] = 0
    as_int(c.v)[page, :, :, 7] = 0x7E  # 448
    q = torch.randn(n, 2, d, device="cuda", dtype=torch.bfloat16)
    scale = 1 / math.sqrt(d)
    o, lse, ran = _attend(c, q, WIDE if n > 1 else 0, scale)
    assert ran == (STREAM if n == 1 else CHUNK)
    k, v = c.sequence("k", 0), c.sequence("v", 0)
    want, want_abs, want_lse = attention(q, k, v, scale, torch.full((n,), 256, device="cuda"))
    if ran == CHUNK:
        assert_attention(o, lse, want, want_abs, want_lse)
        return
    ev = torch.full((256,), -6.0, dtype=torch.float64, device="cuda")
    ev[64:128] += up
    s = q.double().transpose(0, 1) @ k[:, 0].t() * scale  # [2, 1, 256]
    p = torch.exp(s - want_lse[..., None] + ev * math.log(2))  # weights of the stored values
    top = p.amax(-1, keepdim=True)
    low = torch.where(p < 2.0 ** -21 * top, top.expand_as(p), torch.zeros_like(p))
    lost = (low @ torch.ldexp(v[:, 0], -ev[:, None]).abs()).transpose(0, 1)
    err = (o.double() - want).abs()
    print(f"scales {up} powers apart: {float((err / want_abs).max()):.1e} of the summed magnitudes at most")
    assert bool((err <= bound(want, want_abs, lost)).all()), float((err / want_abs).max())
