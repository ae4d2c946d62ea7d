"""Helpers of the paged key-value cache tests: caches whose unused rows hold
NaN, and the definitions in 64 bits, one sequence at a time.

Bounds (half a step of a type relative to the value: bf16 2^-8, fp16 2^-11,
e4m3 2^-4):
- a turned value a cos t -+ b sin t rounded to bf16: 2^-8 |y|, and for the 32-bit
  arithmetic (an angle to 2^-24 turns = 2 pi 2^-24, sine and cosine to two units
  of 2^-24, two products and a sum) less than 2^-20 (|a| + |b|);
- an attention output: the weights w_j enter the product of P and V rounded to
  bf16 (fp16 over an e4m3 cache), at most 2^-8 sum_j w_j |v_j|; the result is
  rounded to bf16, 2^-8 |o|; the 32-bit scores, sums of d = 128 products at most,
  move an exponent by at most 128 * 2^-24 * scale * sum_i |q_i k_i| (below 10 for
  the inputs here), so a weight by less than 2^-13, and the sums of P and of the
  products add less than that again: 2^-12 sum_j w_j |v_j|;
- a log-sum-exp: the same 2^-13, and 2^-22 of its value.
"""

import math

import torch

BF16 = 2.0 ** -8
E4M3 = 2.0 ** -4
E4M3_MAX = 448.0


def as_int(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


class Cache:
    """Sequences of the given lengths in shuffled pages, unused rows NaN."""

    def __init__(self, lens, H_kv, d, page, kind="bf16", spare=2, seed=0, width=None, paired=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.page, self.kind = list(lens), page, kind
        used = [-(-n // page) for n in lens]
        pages = sum(used) + spare
        self.width = max([1] + used) if width is None else width
        dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
        nan = torch.full((), float("nan")).to(dtype)
        if paired:  # keys and values as halves of one tensor
            both = torch.empty(pages, 2, H_kv, page, d, dtype=dtype, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k = torch.empty(pages, H_kv, page, d, dtype=dtype, device="cuda")
            self.v = torch.empty(pages, H_kv, page, d, dtype=dtype, device="cuda")
        self.k_scale = self.v_scale = None
        if kind == "e4m3":
            self.k_scale = 0.01 + 0.02 * torch.rand(H_kv, generator=g, device="cuda")
            self.v_scale = 0.01 + 0.02 * torch.rand(H_kv, generator=g, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda").tolist()
        table = torch.full((len(lens), self.width), -7, dtype=torch.int32)  # entries that nothing reads
        self.ids = []
        for b, n in enumerate(used):
            self.ids.append([order.pop() for _ in range(n)])
            table[b, :n] = torch.tensor(self.ids[b], dtype=torch.int32)
        self.table = table.cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        for t in (self.k, self.v):
            as_int(t).fill_(int(as_int(nan.reshape(1))[0]))
        self.keys, self.values = [], []  # what the sequences hold, in 64 bits
        for b, n in enumerate(lens):
            for cache, scale, kept in ((self.k, self.k_scale, self.keys), (self.v, self.v_scale, self.values)):
                x = torch.randn(n, H_kv, d, generator=g, device="cuda")
                if kind == "e4m3":
                    x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)
                    kept.append(x.double() * scale.double()[:, None])
                else:
                    x = x.to(dtype)
                    kept.append(x.double())
                self.put(cache, b, 0, x)

    def spots(self, b, pos):
        ids = torch.tensor(self.ids[b] or [0], device="cuda")
        return ids[pos // self.page], pos % self.page

    def put(self, cache, b, start, x):
        if x.shape[0]:
            page, row = self.spots(b, torch.arange(start, start + x.shape[0], device="cuda"))
            as_int(cache)[page, :, row] = as_int(x.contiguous())

    def get(self, cache, b, start, n):
        page, row = self.spots(b, torch.arange(start, start + n, device="cuda"))
        return as_int(cache)[page, :, row].contiguous().view(cache.dtype)

    def handle(self):
        from exact_attention_15_gb300 import binding
        return binding.PagedCache(self.k, self.v, k_scale=self.k_scale, v_scale=self.v_scale)


def attention(q, k, v, scale, last):
    """Definition in 64 bits of q [n, H_q, d] over k, v [L, H_kv, d]; row i sees keys
    j < last[i]. Returns o, sum_j w_j |v_j| and lse."""
    n, H_q, d = q.shape
    g = H_q // k.shape[1]
    k, v = k.repeat_interleave(g, 1).transpose(0, 1), v.repeat_interleave(g, 1).transpose(0, 1)
    s = q.double().transpose(0, 1) @ k.transpose(1, 2) * scale  # [H, n, L]
    hidden = torch.arange(k.shape[1], device=q.device)[None] >= last[:, None]
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None])
    return (w @ v).transpose(0, 1), (w @ v.abs()).transpose(0, 1), lse


def assert_attention(o, lse, want, want_abs, want_lse, what=""):
    err = (o.double() - want).abs()
    bound = BF16 * want.abs() + (BF16 + 2.0 ** -12) * want_abs + 1e-30
    assert bool((err <= bound).all()), (what, float((err / bound).max()))
    empty = want_lse == -math.inf
    assert torch.equal(empty, lse == -math.inf), what
    err = (lse.double() - want_lse)[~empty].abs()
    assert bool((err <= 2.0 ** -13 + 2.0 ** -22 * want_lse[~empty].abs()).all()), (what, float(err.max()))


def turned(x, pos, inv_freq, interleaved):
    """Rotary embedding in 64 bits; also |a| + |b| of each value's pair."""
    y, size = x.double().clone(), x.double().abs()
    if inv_freq is None:
        return y, torch.zeros_like(y)
    m = inv_freq.numel()
    i0 = torch.arange(0, 2 * m, 2) if interleaved else torch.arange(m)
    i1 = i0 + (1 if interleaved else m)
    t = pos.double()[:, None, None] * inv_freq.double()
    a, b = y[..., i0].clone(), y[..., i1].clone()
    y[..., i0] = a * t.cos() - b * t.sin()
    y[..., i1] = a * t.sin() + b * t.cos()
    pair = a.abs() + b.abs()
    size = torch.zeros_like(y)
    size[..., i0], size[..., i1] = pair, pair
    return y, size
