"""The bound of attention over an e4m3 cache tells weights of fewer bits from the kernel's:
mistakes planted in the definition, on the CPU."""

import pytest

torch = pytest.importorskip("torch")

from paged_weights import LIFT, SMALL, bound, half_step_bf16, small_weights  # noqa: E402

ROUND = {
    "fp16 at 2^7 of the weight": lambda w: (w * LIFT).half().double() / LIFT,
    "fp16": lambda w: w.half().double(),
    "bf16": lambda w: w.bfloat16().double(),
    "e4m3 at 2^7": lambda w: (w * LIFT).to(torch.float8_e4m3fn).double() / LIFT,
}


def _passes(how, exponent, d):
    w, v = small_weights(exponent, d)
    want = (w[:, None] * v).sum(0) / w.sum()
    got = ((ROUND[how](w)[:, None] * v).sum(0) / w.sum()).bfloat16().double()
    assert float(w.min()) > 2.0 ** -21  # none below the normal numbers
    return bool(((got - want).abs() <= bound(want, want, torch.zeros_like(want))).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("how", ROUND)
def test_bound_tells_weights_of_fewer_bits(how, d):
    passed = [_passes(how, e, d) for e in SMALL]
    assert all(passed) if how == "fp16 at 2^7 of the weight" else not all(passed)


def test_half_step_of_bf16():
    x = torch.tensor([1.0, 1.5, 1.9921875, 2.0, 0.75, -3.0, 0.0], dtype=torch.float64)
    assert half_step_bf16(x).tolist() == [2.0 ** -8] * 3 + [2.0 ** -7, 2.0 ** -9, 2.0 ** -7, 2.0 ** -134]
    y = torch.rand(10000, dtype=torch.float64) * 8
    assert bool(((y.bfloat16().double() - y).abs() <= half_step_bf16(y)).all())
