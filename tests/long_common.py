"""Helpers of the tests of pages with scales of their own, page bounds, page selection
and lists of pages: caches whose unused rows hold NaN, and definitions in 64 bits.

A stored e4m3 x of page p and head h stands for x 2^(byte[p, h] - 127).
"""

import math

import torch

from paged_common import BF16, E4M3_MAX, as_int, attention

E8M0 = torch.float8_e8m0fnu
NAN8 = 0x7F


def values_of(stored, exps):
    """64-bit values of stored e4m3 [..., rows, d] with exponent bytes [...]."""
    return torch.ldexp(stored.double(), exps.double()[..., None, None] - 127)


class Pages:
    """Sequences of the given lengths in shuffled e4m3 pages with a power of two each;
    unused rows are NaN, exponents of unused pages 255."""

    def __init__(self, lens, H_kv, d, page, k_exp=(-8, -4), v_exp=(-8, -4), spare=2, seed=0, width=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.page, self.H_kv, self.d = list(lens), page, H_kv, d
        used = [-(-n // page) for n in lens]
        n_pages = sum(used) + spare
        self.width = max([1] + used) if width is None else width
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        table = torch.full((len(lens), self.width), -7, dtype=torch.int32)  # entries that nothing reads
        self.ids = []
        for b, n in enumerate(used):
            self.ids.append([order.pop() for _ in range(n)])
            table[b, :n] = torch.tensor(self.ids[b], dtype=torch.int32)
        self.table = table.cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.k, self.v, self.k_exp, self.v_exp = [], [], [], []
        for name, (lo, hi) in (("k", k_exp), ("v", v_exp)):
            x = (torch.randn(n_pages, H_kv, page, d, generator=g, device="cuda") * 64).clamp(-E4M3_MAX, E4M3_MAX)
            x = x.to(torch.float8_e4m3fn)
            e = torch.full((n_pages, H_kv), 255, dtype=torch.uint8, device="cuda")
            used_rows = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
            for b, ids in enumerate(self.ids):
                for i, p in enumerate(ids):
                    used_rows[p, :min(page, lens[b] - i * page)] = True
                    e[p] = torch.randint(lo + 127, hi + 128, (H_kv,), generator=g, device="cuda", dtype=torch.uint8)
            as_int(x)[~used_rows[:, None, :, None].expand_as(x)] = NAN8
            setattr(self, name, x)
            setattr(self, name + "_exp", e)

    def handle(self):
        from exact_attention_15_gb300 import binding
        return binding.PagedCache(self.k, self.v, k_scale=self.k_exp.view(E8M0), v_scale=self.v_exp.view(E8M0))

    def sequence(self, name, b):
        """What sequence b holds, [len, H_kv, d] in 64 bits."""
        x, e = getattr(self, name), getattr(self, name + "_exp")
        ids = torch.tensor(self.ids[b] or [0], device="cuda")
        return values_of(x[ids], e[ids]).transpose(1, 2).reshape(-1, self.H_kv, self.d)[:self.lens[b]]

    def attention(self, q, b, scale, last):
        """paged_common.attention over sequence b, its sum of w_j |v_j| with what the weights' fp16 adds.

        The kernel for few tokens holds p_j = w_j 2^ev_j, the weight of the stored value c_j, as fp16 at 2^7 times
        p_j / 2^m or more, m being the largest log2 p so far (less 8 at most, which only raises the
        factor). fp16 rounds to 11 bits, which 2^-12 of |w_j v_j| in assert_attention's bound covers, but
        not below 2^-14: there it moves by half a step of 2^-24, 2^-25. That is 2^-32 of the largest p
        (a later and larger m scales what was summed down, the error with it), so o moves by up to
        2^-32 max_i p_i sum_j |c_j| more. It counts where the c of the largest p is 0 in a column and all the
        other p lie 22 bits and more below."""
        k, v = self.sequence("k", b), self.sequence("v", b)
        o, o_abs, lse = attention(q, k, v, scale, last)
        g, n = q.shape[1] // self.H_kv, k.shape[0]
        if n == 0:
            return o, o_abs, lse
        ids = torch.tensor(self.ids[b], device="cuda")
        ev = (self.v_exp[ids].double() - 127).repeat_interleave(self.page, 0)[:n].t()  # [H_kv, n]
        stored = torch.ldexp(v, -ev.t()[..., None]).abs().sum(0)                         # [H_kv, d]
        s = q.double().transpose(0, 1) @ k.repeat_interleave(g, 1).permute(1, 2, 0) * scale
        s = s.masked_fill(torch.arange(n, device="cuda")[None] >= last[:, None], -math.inf)
        p = (s + ev.repeat_interleave(g, 0)[:, None] * math.log(2)).amax(-1) - lse       # log p, [H_q, rows]
        most = torch.exp(p.nan_to_num(nan=-math.inf)).t()                               # (no key seen: 0)
        return o, o_abs + 2.0 ** -32 * most[..., None] * stored.repeat_interleave(g, 0) / (BF16 + 2.0 ** -12), lse


def exponent(most):
    """The smallest e from -64 to 24 with most <= 448 2^e (24 if there is none)."""
    if not most > 0:
        return -64
    m, x = math.frexp(most)
    return max(-64, min(24, x - 9 + (m > 0.875)))


def encoded(x, e):
    """64-bit values as e4m3 of x / 2^e, rounded once."""
    y = torch.ldexp(x, torch.full_like(x, float(-e))).clamp(-E4M3_MAX, E4M3_MAX)
    # torch rounds 64 bits by way of 32: values are spread enough for that to matter nowhere
    # but within 2^-24 of a border, which the caller's bound allows for
    return y.float().to(torch.float8_e4m3fn)


def bounds_of(k, rows):
    """Minimum and maximum of the first `rows` of k [H_kv, page, d] (64 bits)."""
    x = k[:, :rows]
    return torch.stack((x.amin(1), x.amax(1)), 1)


def scores(q, bounds):
    """Bounds of q . k in 64 bits, the largest over a group: q [H_kv, group, d], bounds
    [n, H_kv, 2, d]. NaN above everything."""
    q, b = q.double(), bounds.double()
    s = torch.einsum("hgd,nhd->hgn", q.clamp(min=0), b[:, :, 1]) + torch.einsum("hgd,nhd->hgn", q.clamp(max=0), b[:, :, 0])
    # an infinity is below a NaN: the largest number stands for the one, infinity for the other
    s = s.clamp(max=torch.finfo(torch.float64).max)
    return torch.where(s.isnan(), torch.full_like(s, math.inf), s).amax(1)  # [H_kv, n]


def selected(q, bounds, ids, seen, page, count, first, last):
    """Page indices [H_kv, count] (-1 behind the last) and keys in them of one token."""
    H_kv = bounds.shape[1]
    n = -(-seen // page)
    out = torch.full((H_kv, count), -1, dtype=torch.int32)
    ids = ids[:n]
    if n <= count:
        out[:, :n] = torch.tensor(ids, dtype=torch.int32)
        return out, seen
    s = scores(q, bounds[torch.tensor(ids, device=bounds.device)])[:, first:n - last].cpu()
    room = count - first - last
    for h in range(H_kv):
        top = torch.sort(s[h], descending=True, stable=True).indices[:room].sort().values + first
        at = list(range(first)) + top.tolist() + list(range(n - last, n))
        out[h] = torch.tensor([ids[i] for i in at], dtype=torch.int32)
    return out, seen - (n - count) * page
