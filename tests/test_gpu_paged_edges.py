"""The paged key-value cache at the ends of its range."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from exact_attention_15_gb300 import binding  # noqa: E402
from paged_common import E4M3_MAX, Cache  # noqa: E402


@pytest.fixture(autouse=True)
def _clean():
    assert binding.attn_check(None) == 0
    yield
    assert binding.attn_check(None) == 0


def _offsets(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


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
