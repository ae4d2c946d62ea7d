"""Weights over an e4m3 cache, whose product with the values takes them as fp16 at 2^7
times their value: the bound of an output that this gives, and inputs on which weights of
fewer bits pass it.

Bound of an output o = sum_j w_j v_j / sum_j w_j, the weights taken relative to the largest
(the bias that the kernel subtracts lies at most that high, so that its weights are no
smaller than these):
- a weight rounded to fp16 at 2^7 times its value: half a step of 11 bits, 2^-11 of it,
  where that is a normal number (from 2^-21 on), else half a step of 2^-24 / 2^7, 2^-32;
- the 32-bit scores, exponentials and sums: 2^-12 as in ``paged_common``;
- the result rounded to bf16: half a step between its neighbours.
"""

import math

import torch

LIFT = 2.0 ** 7


def half_step_bf16(x):
    """Half the distance between bf16's values at |x| (8 bits, none below 2^-133)."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -126))
    return torch.ldexp(torch.ones_like(x), e - 9)


def bound(want, want_abs, lost):
    """want_abs: sum_j w_j |v_j| / sum_j w_j; lost: sum of |v_j| over the weights below 2^-21
    / sum_j w_j."""
    inner = (2.0 ** -11 + 2.0 ** -12) * want_abs + 2.0 ** -32 * lost
    return inner + half_step_bf16(want.abs() + inner)


# Exponents of a small weight. 2^-20.5 is 11.3 of fp16's smallest steps, and stays within
# 2^-11 of itself only when lifted. The other lies just between two of bf16's values.
SMALL = (20.5, 20 - math.log2(1 + 2.0 ** -8))


def small_weights(exponent, d, seed=0):
    """200 keys: every 16th with weight 1 and no value, the others with weight
    2^-exponent and values 0.5 to 3.5. Returns the weights and the values [200, d], in 64
    bits. (Every 16th: each warp of the streaming kernel takes 16 keys of a tile and keeps a
    bias of its own.)"""
    g = torch.Generator().manual_seed(seed)
    w = torch.full((200,), 2.0 ** -exponent, dtype=torch.float64)
    v = 0.5 * torch.randint(1, 8, (200, d), generator=g).double()
    w[::16], v[::16] = 1.0, 0.0
    return w, v
