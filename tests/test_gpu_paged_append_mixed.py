"""Appending to pages with scales where the mean of the new tokens decides between the kernels: on both sides
of the border, and batches of a prompt among single tokens, against the definition in 64 bits."""

import pytest

torch = pytest.importorskip("torch")

from long_common import Pages  # noqa: E402
from test_gpu_paged_pages import _append  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H_q,H_kv,d,page,rotary,interleaved", [
    (8, 2, 128, 16, 128, False), (6, 3, 64, 32, 32, True), (0, 1, 128, 256, 64, False), (4, 2, 128, 64, 0, False)])
@pytest.mark.parametrize("new,ctx", [
    ([24, 24, 24], [0, 40, 300]), ([25, 24, 24], [7, 0, 255]), ([17], [250]), ([33, 2], [31, 0]),
    ([300] + [1] * 12, [5] + list(range(12, 24))), ([300] + [1] * 8, [0] + list(range(60, 68)))],
    ids=["24", "above 24", "17", "33 and 2", "prompt among 12", "prompt among 8"])
def test_append_by_the_mean(new, ctx, H_q, H_kv, d, page, rotary, interleaved):
    lens = [n + x for n, x in zip(new, ctx)]
    c = Pages(lens, H_kv, d, page, (-9, -3), (-9, -3), seed=sum(lens))
    _append(c, new, H_q, rotary, interleaved, fused=bool(sum(new) & 1))
