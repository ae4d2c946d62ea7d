"""Cases of the operators for long contexts over the paged key-value cache:

append   new tokens into an e4m3 cache with a power-of-two scale for each page and KV
         head (with the rotary position embedding on the way)
attend   attention of one new token per sequence, or of packed chunks, over such a cache
bounds   elementwise minimum and maximum of the keys of the pages that new tokens touched
select   the pages that each query token attends to, for every KV head: those with the
         largest upper bound of q . k, besides the first and the last ones
lists    attention of one token per sequence over such lists of pages

Cache layout: k and v are [num_pages, H_kv, page_size, d]; position t of sequence b lies in
page page_table[b, t // page_size], row t % page_size. seq_lens[b] is the length of sequence
b with its new tokens; new token i of n is at position seq_lens[b] - n + i. The scales are
exponents plus 127 in bytes [num_pages, H_kv]: a stored x stands for x 2^(byte - 127).

Exponents: E(M) is the smallest e from -64 to 64 with M <= 448 2^e (64 if there is none). A
page that begins with a new token takes E of the largest finite magnitude among its new
values of that head; another one the larger of that and what it had, and if it grows the
rows that it holds are encoded again. Keys that are turned count with 1.5 times their
magnitude before the turn (a turned element is at most sqrt 2 of it).

``own`` selects the framework's kernels or the plain torch forms.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
E_MOST = 64


def listed():
    return [
        # one decoding step of a large batch
        dict(name="append_step", op="append", B=256, new_lo=1, new_hi=1, ctx_lo=17, ctx_hi=2048, H_q=32, H_kv=8, d=128, page=32,
             rotary=64, interleaved=True, lens=1),
        # the prompts of a ragged batch, projected in one fused matrix product
        dict(name="append_prompts", op="append", B=16, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, H_q=32, H_kv=8, d=128, page=64,
             rotary=128, interleaved=False, lens=2),
        # a single user with a short context: latency
        dict(name="attend_one_short", op="attend", B=1, ctx_lo=777, ctx_hi=777, H_q=32, H_kv=8, d=128, page=16, lens=3),
        # a serving batch of ragged contexts
        dict(name="attend_batch", op="attend", B=64, ctx_lo=1024, ctx_hi=16384, H_q=32, H_kv=8, d=128, page=64, lens=4),
        # a few drafted tokens per sequence are verified against long contexts
        dict(name="attend_drafted", op="attend", B=8, new_lo=4, new_hi=4, ctx_lo=2000, ctx_hi=16000, H_q=32, H_kv=8, d=128, page=32,
             causal=True, lens=5),
        # the prompts of a ragged batch, nothing in the cache before them
        dict(name="attend_prompts", op="attend", B=8, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, H_q=32, H_kv=8, d=128, page=64,
             causal=True, lens=6),
        # a decoding step of a serving batch: the bounds of the pages being filled
        dict(name="bounds_step", op="bounds", B=64, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=32768, H_q=32, H_kv=8, d=128, page=64,
             kind="paged", lens=7),
        # all bounds of the prompts of a ragged batch
        dict(name="bounds_prompts", op="bounds", B=16, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, H_q=32, H_kv=8, d=128, page=32,
             kind="bf16", lens=8),
        # a single user with a long context
        dict(name="select_one_long", op="select", B=1, new_lo=1, new_hi=1, ctx_lo=131071, ctx_hi=131071, H_q=32, H_kv=8, d=128, page=32,
             count=64, first=1, last=2, lens=9),
        # a serving batch of ragged long contexts
        dict(name="select_batch", op="select", B=64, new_lo=1, new_hi=1, ctx_lo=4096, ctx_hi=32768, H_q=32, H_kv=8, d=128, page=64,
             count=32, first=1, last=1, lens=10),
        # a single user: 2048 of the keys of a long context
        dict(name="lists_one", op="lists", B=1, H_q=32, H_kv=8, d=128, page=32, count=64, kind="paged", spread=64, lens=11),
        # a serving batch, 2048 keys a token and head
        dict(name="lists_batch", op="lists", B=64, H_q=32, H_kv=8, d=128, page=64, count=32, kind="bf16", spread=8, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:  # no more than the largest listed case of its operator
        case = _drawn(rng)
        cost = work(case)
        if all(cost[x] <= max(work(c)[x] for c in listed() if c["op"] == case["op"]) for x in cost):
            return case


def _drawn(rng):
    op = rng.choice(["append", "attend", "bounds", "select", "lists"])
    H_kv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, H_kv=H_kv, H_q=H_kv * rng.choice([1, 2, 4, 5, 8] if H_kv <= 8 else [1, 2]), d=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), lens=rng.randrange(1 << 20))
    row = H_kv * c["d"]
    if op in ("append", "bounds"):
        c["B"] = _log(rng, 1, 256)
        hi = min(4096, max(1, (24000 if op == "append" else 16000) * 6144 // ((c["H_q"] + 2 * H_kv) * c["d"]) // c["B"]))
        c["new_hi"] = 1 if rng.random() < 0.4 else _log(rng, 1, hi)
        c["new_lo"] = 1 + (c["new_hi"] - 1) // 3
        c["ctx_hi"] = rng.choice([0, _log(rng, 1, 2048)])
        c["ctx_lo"] = c["ctx_hi"] // 4
        if op == "bounds":
            c["kind"] = rng.choice(["bf16", "e4m3", "paged"])
        else:
            c["rotary"] = rng.choice([0, c["d"], c["d"] // 2])
            c["interleaved"] = rng.random() < 0.5
    elif op == "attend" and rng.random() < 0.5:  # a decoding step
        c["B"] = _log(rng, 1, 256)
        hi = max(2, min(131072, 300_000 * 1024 // row // c["B"]))
        c["ctx_hi"] = _log(rng, 1, hi)
        c["ctx_lo"] = max(1, c["ctx_hi"] // rng.choice([1, 2, 8, 64]))
    elif op == "attend":
        c["B"] = _log(rng, 1, 16)
        most = 1_700_000_000 // (c["B"] * c["H_q"])  # scores of one head that the plain form holds
        c["new_hi"] = _log(rng, 1, min(4096, int(math.sqrt(most))))
        c["new_lo"] = 1 + (c["new_hi"] - 1) // rng.choice([1, 4])
        room = min(32768, most // c["new_hi"]) - c["new_hi"]
        c["ctx_hi"] = 0 if room < 2 or rng.random() < 0.3 else _log(rng, 1, room)
        c["ctx_lo"] = c["ctx_hi"] // 2
        c["causal"] = rng.random() < 0.8
    elif op == "select":
        c["B"] = _log(rng, 1, 128)
        c["new_hi"] = rng.choice([1, 1, 1, 2, 4, 7])
        c["new_lo"] = 1 + (c["new_hi"] - 1) // 3
        blocks = max(2, min(8192, 60_000_000 // (c["B"] * c["new_hi"] * max(2 * row, c["H_q"] * c["d"] // 2))))
        c["ctx_hi"] = _log(rng, 1, blocks * c["page"])
        c["ctx_lo"] = max(1, c["ctx_hi"] // rng.choice([1, 2, 8]))
        c["first"], c["last"] = rng.choice([0, 1, 2]), rng.choice([1, 2, 3])
        c["count"] = _log(rng, c["first"] + c["last"], 128)
    else:
        c["B"] = _log(rng, 1, 128)
        c["count"] = _log(rng, 1, max(1, min(256, 100_000_000 // (c["B"] * row * c["page"]))))
        c["kind"] = rng.choice(["bf16", "e4m3", "paged"])
        c["spread"] = rng.choice([1, 4, 16])
    return c


def _lengths(case):
    """New tokens and total length of each sequence: the same for every seed."""
    r = random.Random(case["lens"])
    B = case["B"]
    if case["op"] == "lists":  # keys of the lists: whole pages and the last one's
        return [1] * B, [(case["count"] - 1) * case["page"] + r.randint(1, case["page"]) for _ in range(B)]
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 1 for _ in range(B)]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(B)]
    # the range of a decoding step that attends is that of whole lengths
    return new, (ctx if "new_lo" not in case else [n + c for n, c in zip(new, ctx)])


def _as_int(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def _inputs(case, seed):
    """Everything on the GPU that a call takes, from the seed alone."""
    dev, op = "cuda", case["op"]
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    new, total = _lengths(case)
    B, H_q, H_kv, d, page = (case[x] for x in ("B", "H_q", "H_kv", "d", "page"))
    T = sum(new)
    kind = case.get("kind", "bf16" if op == "select" else "paged")
    s = dict(case=case, kind=kind, lens=torch.tensor(total, dtype=torch.int32, device=dev))
    if op == "lists":
        # what a selection leaves: the cache is `spread` times what the lists name
        pages = B * case["count"] * case["spread"] + 3
        weight = torch.rand(B, H_kv, case["count"] * case["spread"], generator=g, device=dev)
        at = weight.topk(case["count"], dim=2).indices.sort(dim=2).values + torch.arange(B, device=dev)[:, None, None] * (
            case["count"] * case["spread"])
        s["table"] = torch.randperm(pages, generator=g, device=dev)[at].to(torch.int32).contiguous()
    else:
        width = max(1, -(-max(total) // page))
        pages = sum(-(-n // page) for n in total) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(B, width, dtype=torch.int32)
        at = 0
        for b, n in enumerate(total):
            m = -(-n // page)
            table[b, :m] = torch.arange(at, at + m, dtype=torch.int32)
            at += m
        s["table"] = order[table.to(dev).long()].contiguous()
    for name in ("k", "v"):
        s[name + "_scale"] = s[name + "_exp"] = None
        if op == "select":  # the bounds alone are read
            s[name] = torch.empty(pages, H_kv, page, d, dtype=torch.bfloat16, device=dev)
            continue
        x = normal(pages, H_kv, page, d)
        if kind == "e4m3":  # scales that use a good part of e4m3's range
            s[name + "_scale"] = 0.01 + 0.01 * torch.rand(H_kv, generator=g, device=dev)
        elif kind == "paged":  # pages of values of different sizes, from about 2^-4 to 2^4
            s[name + "_exp"] = torch.randint(127 - 11, 127 - 3, (pages, H_kv), generator=g, device=dev, dtype=torch.uint8)
            if op == "append":  # of values like the new ones, one page in eight of smaller ones
                s[name + "_exp"] = (127 - 6 - (s[name + "_exp"] == 127 - 11).to(torch.uint8)).contiguous()
        s[name] = x if kind == "bf16" else (x * 64).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    if op == "append":
        x = normal(T, H_q + 2 * H_kv, d)  # views of one projection's output
        s["q"], s["new_k"], s["new_v"] = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        half = case["rotary"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(dev) if half else None
    elif op != "bounds":
        s["q"] = normal(T, H_q, d)
    if op in ("bounds", "select"):
        # as of keys that drift from page to page
        mid = normal(pages, H_kv, d)
        s["bounds"] = torch.stack((mid - normal(pages, H_kv, d).abs() - 1, mid + normal(pages, H_kv, d).abs() + 1), 2)
    s["cu"] = None
    if "new_lo" in case and (op == "attend" or case["new_hi"] > 1):
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev)
    s["tokens"], s["most_new"] = T, max(new)  # a program that packs its batch knows its tokens and its longest piece
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from exact_attention_15_gb300 import binding
        scales = [s[x + "_exp"].view(torch.float8_e8m0fnu) if s[x + "_exp"] is not None else s[x + "_scale"] for x in ("k", "v")]
        s["cache"] = binding.PagedCache(s["k"], s["v"], k_scale=scales[0], v_scale=scales[1])
    return s


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "bounds": _plain_bounds, "select": _plain_select,
                "lists": _plain_lists}[op](s)
    from exact_attention_15_gb300 import binding
    if op == "append":
        q = binding.paged_append(s["cache"], s["q"], s["new_k"], s["new_v"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                 inv_freq=s["inv_freq"], interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if op == "bounds":
        return binding.paged_bounds(s["cache"], s["bounds"], s["table"], s["lens"], cu_seqlens=s["cu"], tokens=s["tokens"])
    if op == "select":
        pages, lens = binding.paged_select(s["cache"], s["q"], s["bounds"], s["table"], s["lens"], c["count"], cu_seqlens=s["cu"],
                                           keep_first=c["first"], keep_last=c["last"])
        return {"pages": pages, "lens": lens}
    if s["cu"] is None:
        o, lse = binding.paged_decode(s["cache"], s["q"], s["table"], s["lens"])
    else:
        o, lse = binding.paged_forward(s["cache"], s["q"], s["table"], s["lens"], s["cu"], causal=c["causal"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ plain forms

def _power(e):
    """2^e in fp32, e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _where_new(s):
    """Offsets, and sequence, place in its chunk and position of every new token."""
    B, dev = s["case"]["B"], s["lens"].device
    T = s["q"].shape[0]
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=dev)
    t = torch.arange(T, device=dev)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    place = t - cu[seq]
    pos = s["lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + place
    return cu, seq, place, pos


def _rotated(x, pos, inv_freq, interleaved):
    x = x.float()
    if inv_freq is None:
        return x
    angle = pos.double()[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = inv_freq.shape[0]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _exponent(most):
    """The smallest e from -64 to 64 with most <= 448 2^e = 0.875 2^(e + 9)."""
    m, x = torch.frexp(most)
    e = x - 9 + (m > 0.875)
    return torch.where(most == 0, torch.full_like(e, -E_MOST), e).clamp(-E_MOST, E_MOST)


def _encoded(x, e):
    return (x * _power(-e)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append(s):
    c = s["case"]
    B, H_kv, size = c["B"], c["H_kv"], c["page"]
    cu, seq, _, pos = _where_new(s)
    table, dev = s["table"].long(), pos.device
    n = cu[1:] - cu[:-1]
    start = s["lens"].long() - n  # position of each sequence's first new token
    touched = (s["most_new"] + size - 2) // size + 1  # pages of a sequence at most
    place = pos // size - (start // size)[seq]
    page, row = table[seq, pos // size], pos % size
    unit = seq * touched + place
    every = (start // size)[:, None] + torch.arange(touched, device=dev)
    last = ((start + n - 1) // size)[:, None]
    ids = table[torch.arange(B, device=dev)[:, None], torch.minimum(every, last)]  # [B, touched]
    held = torch.where(every * size >= start[:, None], 0, start[:, None] - every * size)  # rows in use before the call
    turn = s["inv_freq"] is not None
    for name, x, turned in (("k", s["new_k"], turn), ("v", s["new_v"], False)):
        size_of = x.float().abs()
        size_of = torch.where(size_of < math.inf, size_of, torch.zeros_like(size_of)).amax(-1) * (1.5 if turned else 1.0)
        most = torch.zeros(B * touched, H_kv, device=dev).scatter_reduce_(0, unit[:, None].expand(-1, H_kv), size_of, "amax")
        exps, cache = s[name + "_exp"], s[name]
        e = _exponent(most).view(B, touched, H_kv)
        old = exps[ids].to(torch.int32) - 127
        e = torch.where((held > 0)[..., None], torch.maximum(e, old), e)
        # the page that the first new token goes to holds rows already
        kept = _as_int(cache)[ids[:, 0]]
        again = _encoded(kept.view(cache.dtype).float() * _power(old[:, 0])[..., None, None], e[:, 0][..., None, None]).view(torch.uint8)
        mine = (torch.arange(size, device=dev) < held[:, :1])[:, None, :, None]
        _as_int(cache)[ids[:, 0]] = torch.where(mine, again, kept)
        # (places behind a sequence's last page name that one again)
        e = torch.take_along_dim(e, (torch.minimum(every, last) - every[:, :1])[..., None], 1)
        exps[ids] = (e + 127).to(torch.uint8)
        y = _rotated(x, pos, s["inv_freq"], c["interleaved"]) if turned else x.float()
        _as_int(cache)[page, :, row] = _encoded(y, e.flatten(0, 1)[unit][..., None]).view(torch.uint8)
    q = _rotated(s["q"], pos, s["inv_freq"], c["interleaved"]).to(torch.bfloat16)
    return {"q": q, "k": s["k"], "v": s["v"], "k_exp": s["k_exp"], "v_exp": s["v_exp"]}


def _scaled(s, name, pages, heads=None):
    """The values of the pages in fp32 (of every head, or of the given one for each page)."""
    cache, scale, exps = s[name], s[name + "_scale"], s[name + "_exp"]
    at = (pages,) if heads is None else (pages, heads)
    x = _as_int(cache)[at].view(cache.dtype).float()
    if exps is not None:
        x = x * _power(exps[at].to(torch.int32) - 127)[..., None, None]
    elif scale is not None:
        x = x * (scale if heads is None else scale[heads])[..., None, None]
    return x


def _gathered(s, name):
    """The sequences' keys or values, [B, H_kv, L, d] in fp32."""
    table = s["table"].long()
    if table.dim() == 3:
        return _scaled(s, name, table, torch.arange(table.shape[1], device=table.device)[:, None]).flatten(2, 3)
    return _scaled(s, name, table).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _softmax_product(scores, hidden, values):
    """Output and log-sum-exp of the scores that are not hidden; rows without any give 0 and -inf."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    return o, (top + total.log()).squeeze(-1)


def _plain_lists(s):
    c = s["case"]
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    past = torch.arange(k.shape[2], device=k.device)[None, :] >= s["lens"][:, None]
    scores = torch.matmul(s["q"].float().view(B, H_kv, H_q // H_kv, d), k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    o, lse = _softmax_product(scores, past[:, None, None, :], v)
    return {"o": o.reshape(B, H_q, d).to(torch.bfloat16), "lse": lse.reshape(B, H_q)}


def _plain_attend(s):
    if s["cu"] is None:
        return _plain_lists(s)
    c = s["case"]
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    n, group = s["most_new"], H_q // H_kv
    cu, seq, place, _ = _where_new(s)
    rows = (cu[:-1, None] + torch.arange(n, device=cu.device)).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, H_kv, group, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, group * n, d)
    k, v = _gathered(s, "k"), _gathered(s, "v")
    key = torch.arange(k.shape[2], device=k.device)
    last = s["lens"].long()[:, None] - 1  # the last key that each new token sees
    if c["causal"]:
        last = last - (cu[1:] - cu[:-1])[:, None] + 1 + torch.arange(n, device=k.device)
    hidden = (key[None, None, :] > last[:, :, None]).expand(B, n, key.numel())
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, H_kv, group, n, -1)
    o, lse = _softmax_product(scores, hidden[:, None, None], v[:, :, None])
    o = o.reshape(B, H_q, n, d)[seq, :, place]
    return {"o": o.to(torch.bfloat16), "lse": lse.reshape(B, H_q, n)[seq, :, place].t().contiguous()}


def _plain_bounds(s):
    c = s["case"]
    B, size, dev = c["B"], c["page"], s["lens"].device
    lens = s["lens"].long()
    n = (s["cu"][1:] - s["cu"][:-1]).long() if s["cu"] is not None else torch.ones_like(lens)
    first, last = (lens - n) // size, (lens - 1) // size
    touched = (s["most_new"] + size - 2) // size + 1
    place = torch.minimum(first[:, None] + torch.arange(touched, device=dev), last[:, None])
    ids = s["table"].long()[torch.arange(B, device=dev)[:, None], place].flatten()
    free = (torch.arange(size, device=dev) >= (lens[:, None] - place * size).flatten()[:, None])[:, None, :, None]
    k = _scaled(s, "k", ids)
    lo, hi = k.masked_fill(free, math.inf).amin(2), k.masked_fill_(free, -math.inf).amax(2)
    s["bounds"][ids] = torch.stack((lo, hi), 2).to(torch.bfloat16)
    return s["bounds"]


def _plain_select(s):
    """In 64 bits: which pages are chosen hangs on scores next to one another."""
    c = s["case"]
    H_kv, d, size, count = c["H_kv"], c["d"], c["page"], c["count"]
    _, seq, _, pos = _where_new(s)
    table, dev, T = s["table"].long()[seq], pos.device, pos.numel()
    lens = pos + 1
    blocks = (lens + size - 1) // size
    q = s["q"].double().view(T, H_kv, -1, d)
    b = s["bounds"].double()[table].transpose(1, 2)  # [T, H_kv, width, 2, d]
    score = torch.matmul(q.clamp_min(0), b[..., 1, :].transpose(2, 3)) + torch.matmul(q.clamp_max(0), b[..., 0, :].transpose(2, 3))
    score = score.amax(2)  # [T, H_kv, width]
    at = torch.arange(table.shape[1], device=dev)
    kept = (at < c["first"]) | (at >= blocks[:, None] - c["last"])
    score.masked_fill_(kept[:, None], math.inf).masked_fill_((at >= blocks[:, None])[:, None], -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices[..., :count]
    order = torch.nn.functional.pad(order, (0, count - order.shape[2]), value=table.shape[1])
    chosen = torch.minimum(blocks, torch.full_like(blocks, count))
    none = torch.arange(count, device=dev) >= chosen[:, None]
    order = order.masked_fill(none[:, None], table.shape[1]).sort(dim=2).values
    pages = torch.take_along_dim(table[:, None], order.clamp(max=table.shape[1] - 1), 2).masked_fill(none[:, None], -1)
    return {"pages": pages.to(torch.int32), "lens": (lens - (blocks - chosen) * size).to(torch.int32)}


# ------------------------------------------------------------------ definition in 64 bits

def _values(s, name, ids, heads=slice(None)):
    """Pages `ids` in 64 bits."""
    x = _as_int(s[name])[ids, heads].view(s[name].dtype).double()
    if s[name + "_exp"] is not None:
        return torch.ldexp(x, s[name + "_exp"][ids, heads].double()[..., None, None] - 127)
    if s[name + "_scale"] is not None:
        return x * s[name + "_scale"].double()[heads][..., None, None]
    return x


def _exact_append(case, s, new, total):
    freq, size = s["inv_freq"], case["page"]
    pairs = case["rotary"] // 2
    i0 = torch.arange(0, 2 * pairs, 2, device="cuda") if case["interleaved"] else torch.arange(pairs, device="cuda")
    i1 = i0 + (1 if case["interleaved"] else pairs)
    out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double(), "k_exp": s["k_exp"].clone(), "v_exp": s["v_exp"].clone()}
    ids = s["table"].tolist()
    t0 = 0
    for b, n in enumerate(new):
        pos = torch.arange(total[b] - n, total[b], device="cuda")
        x = {"q": s["q"][t0:t0 + n].double(), "k": s["new_k"][t0:t0 + n].double(), "v": s["new_v"][t0:t0 + n].double()}
        large = {"k": x["k"].abs().amax(2) * (1.5 if pairs else 1.0), "v": x["v"].abs().amax(2)}
        if pairs:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None].double() * freq)[:, None, :]
            for name in ("q", "k"):
                z = torch.complex(x[name][..., i0], x[name][..., i1]) * turn
                x[name][..., i0], x[name][..., i1] = z.real, z.imag
        out["q"][t0:t0 + n] = x["q"]
        begin = total[b] - n
        for i in range(begin // size, (total[b] - 1) // size + 1):
            id, r0 = ids[b][i], max(0, begin - i * size)
            lo, hi = max(0, i * size - begin), min(n, (i + 1) * size - begin)
            for name in ("k", "v"):
                e = torch.ceil(torch.log2(large[name][lo:hi].amax(0) / E4M3_MAX))
                # log2 may round at a power of two: the definition is a comparison
                e = torch.where(torch.ldexp(torch.full_like(e, E4M3_MAX), e - 1) >= large[name][lo:hi].amax(0), e - 1, e)
                e = torch.where(torch.ldexp(torch.full_like(e, E4M3_MAX), e) < large[name][lo:hi].amax(0), e + 1, e)
                e = e.clamp(-E_MOST, E_MOST)
                if r0:
                    before = s[name + "_exp"][id].double() - 127
                    e = torch.maximum(e, before)
                    out[name][id][:, :r0] = torch.ldexp(out[name][id][:, :r0], (before - e)[:, None, None])
                y = torch.ldexp(x[name][lo:hi].transpose(0, 1), -e[:, None, None])
                out[name][id][:, r0:r0 + hi - lo] = y.clamp(-E4M3_MAX, E4M3_MAX)
                out[name + "_exp"][id] = (e + 127).to(torch.uint8)
        t0 += n
    return out


def exact(case, seed):
    """One sequence at a time, in 64 bits."""
    s = _inputs(case, seed)
    new, total = _lengths(case)
    op, size, d, H_kv = case["op"], case["page"], case["d"], case["H_kv"]
    group = case["H_q"] // H_kv
    if op == "append":
        return _exact_append(case, s, new, total)
    if op == "bounds":
        out = s["bounds"].double()
        for b, n in enumerate(new):
            for i in range((total[b] - n) // size, (total[b] - 1) // size + 1):
                id = int(s["table"][b, i])
                x = _values(s, "k", id)[:, :total[b] - i * size]
                out[id, :, 0], out[id, :, 1] = x.min(1).values, x.max(1).values
        return out
    if op == "select":
        pages = torch.full((sum(new), H_kv, case["count"]), -1, dtype=torch.int32, device="cuda")
        lens, t = [], 0
        for b, n in enumerate(new):
            for i in range(n):
                seen = total[b] - n + i + 1
                m = -(-seen // size)
                ids = s["table"][b, :m].long()
                box = s["bounds"][ids].double()  # [m, H_kv, 2, d]
                q = s["q"][t].double().view(H_kv, group, d)
                best = torch.stack([torch.maximum(q[:, j] * box[:, :, 0], q[:, j] * box[:, :, 1]).sum(-1) for j in range(group)]).amax(0)
                if m > case["count"]:
                    inner = range(case["first"], m - case["last"])
                    room = case["count"] - case["first"] - case["last"]
                    value = best[inner.start:inner.stop].t().cpu().numpy()
                    for h in range(H_kv):
                        top = sorted((-value[h]).argsort(kind="stable")[:room] + case["first"])
                        at = list(range(case["first"])) + top + list(range(m - case["last"], m))
                        pages[t, h] = ids[torch.tensor(at, device="cuda")].int()
                else:
                    pages[t, :, :m] = ids.int()
                lens.append(seen - max(0, m - case["count"]) * size)
                t += 1
        return {"pages": pages, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    o, lse, t0 = [], [], 0
    for b, n in enumerate(new):
        L = total[b]
        m = -(-L // size)
        kv = []
        for name in ("k", "v"):
            if op == "lists":
                x = torch.stack([_values(s, name, s["table"][b, h, :m].long(), h) for h in range(H_kv)], 1)
            else:
                x = _values(s, name, s["table"][b, :m].long())
            kv.append(x.transpose(1, 2).reshape(-1, H_kv, d)[:L].repeat_interleave(group, dim=1).transpose(0, 1))
        q = s["q"][t0:t0 + n].double().transpose(0, 1)
        w = q @ kv[0].transpose(1, 2) / math.sqrt(d)
        if case.get("causal"):
            w += torch.full((n, L), -math.inf, dtype=torch.float64, device="cuda").triu(L - n + 1)
        lse.append(torch.logsumexp(w, -1))
        o.append((torch.softmax(w, -1) @ kv[1]).transpose(0, 1))
        t0 += n
    return {"o": torch.cat(o), "lse": torch.cat(lse, dim=1) if s["cu"] is not None else torch.stack(lse).squeeze(-1)}


def work(case):
    new, total = _lengths(case)
    op, H_q, H_kv, d, page = (case[x] for x in ("op", "H_q", "H_kv", "d", "page"))
    T, L = sum(new), sum(total)
    if op == "append":
        return {"bytes": T * ((2 * H_q + 2 * H_kv) * d * 2 + 2 * H_kv * d), "flops": 3 * T * (H_q + H_kv) * case["rotary"]}
    size = 2 if case.get("kind") == "bf16" else 1
    if op == "bounds":
        pages = [(n, (n - m) // page) for n, m in zip(total, new)]  # length, first page touched
        keys = sum(n - p * page for n, p in pages)
        return {"bytes": keys * H_kv * d * size + sum(-(-n // page) - p for n, p in pages) * H_kv * 4 * d, "flops": 2 * keys * H_kv * d}
    if op == "select":
        boxes = [-(-n // page) if -(-n // page) > case["count"] else 0 for n in total]
        return {"bytes": sum(boxes) * H_kv * 4 * d + T * H_q * d * 2 + T * H_kv * case["count"] * 4,
                "flops": sum(m * n for m, n in zip(boxes, new)) * 4 * d * H_q}
    seen = sum(n * t - (n * (n - 1) // 2 if case.get("causal") else 0) for n, t in zip(new, total))
    # keys and values once, queries once, outputs and log-sum-exp once
    return {"bytes": 2 * L * H_kv * d * size + T * H_q * (4 * d + 4), "flops": 4 * seen * H_q * d}
