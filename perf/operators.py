"""Cases of the paged key-value cache operators: appending new tokens (with the
rotary position embedding applied on the way), attention of one new token per
sequence, and attention of a packed chunk of new tokens, both over the cache.

Cache layout: k and v are [num_pages, H_kv, page_size, d] in bf16 or e4m3 (with
one fp32 scale per KV head); position t of sequence b lies in page
page_table[b, t // page_size], row t % page_size. seq_lens[b] is the length of
sequence b with its new tokens; new token i of n is at position seq_lens[b] - n + i.

``own`` selects the framework's kernels or the plain torch forms.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # one decoding step of a single user: latency of the smallest append
        dict(name="append_one_token", op="append", B=1, new_lo=1, new_hi=1, ctx_lo=700, ctx_hi=700, H_q=32, H_kv=8, d=128,
             page=16, kind="bf16", rotary=128, interleaved=False, fused=True, lens=1),
        # one decoding step of a large batch into a quantised cache
        dict(name="append_batch_e4m3", op="append", B=256, new_lo=1, new_hi=1, ctx_lo=17, ctx_hi=2048, H_q=32, H_kv=8, d=128,
             page=32, kind="e4m3", rotary=64, interleaved=True, fused=True, lens=2),
        # the prompts of a ragged batch, projected in one fused matrix product
        dict(name="append_prompts", op="append", B=16, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, H_q=32, H_kv=8, d=128,
             page=64, kind="bf16", rotary=128, interleaved=False, fused=True, lens=3),
        # a single user with a short context: latency
        dict(name="decode_one_short", op="decode", B=1, ctx_lo=777, ctx_hi=777, H_q=32, H_kv=8, d=128, page=16, kind="bf16", lens=4),
        # a single user with a long context: the cache's length split over the GPU
        dict(name="decode_one_long", op="decode", B=1, ctx_lo=131071, ctx_hi=131071, H_q=32, H_kv=8, d=128, page=128, kind="bf16", lens=5),
        # a serving batch of ragged contexts, the largest step
        dict(name="decode_batch", op="decode", B=64, ctx_lo=1024, ctx_hi=16384, H_q=32, H_kv=8, d=128, page=64, kind="bf16", lens=6),
        # a large batch over a quantised cache
        dict(name="decode_batch_e4m3", op="decode", B=128, ctx_lo=64, ctx_hi=4096, H_q=32, H_kv=4, d=128, page=32, kind="e4m3", lens=7),
        # heads of 64, no sharing of key-value heads, some sequences just begun
        dict(name="decode_heads_of_64", op="decode", B=32, ctx_lo=1, ctx_hi=2048, H_q=16, H_kv=16, d=64, page=16, kind="bf16", lens=8),
        # a few drafted tokens per sequence are verified against long contexts
        dict(name="chunk_verify", op="chunk", B=8, new_lo=4, new_hi=4, ctx_lo=2000, ctx_hi=16000, H_q=32, H_kv=8, d=128, page=16,
             causal=True, lens=9),
        # the prompts of a ragged batch, nothing in the cache before them
        dict(name="chunk_prompts", op="chunk", B=8, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, H_q=32, H_kv=8, d=128, page=64,
             causal=True, lens=10),
        # the next chunk of two long prompts
        dict(name="chunk_of_long", op="chunk", B=2, new_lo=1024, new_hi=1024, ctx_lo=16000, ctx_hi=31744, H_q=32, H_kv=8, d=128, page=128,
             causal=True, lens=11),
        # short odd prompts with heads of 64
        dict(name="chunk_heads_of_64", op="chunk", B=16, new_lo=33, new_hi=1000, ctx_lo=0, ctx_hi=500, H_q=16, H_kv=16, d=64, page=32,
             causal=True, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "chunk"])
    H_kv = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=op, H_kv=H_kv, H_q=H_kv * rng.choice([1, 2, 4, 5, 8] if H_kv <= 8 else [1, 2]), d=rng.choice([64, 128]),
             page=rng.choice([16, 32, 64, 128]), lens=rng.randrange(1 << 20))
    row = H_kv * c["d"]
    if op == "append":
        c["B"] = _log(rng, 1, 256)
        hi = min(4096, max(1, 24000 * 6144 // ((c["H_q"] + 2 * H_kv) * c["d"]) // c["B"]))
        c["new_hi"] = 1 if rng.random() < 0.4 else _log(rng, 1, hi)
        c["new_lo"] = 1 + (c["new_hi"] - 1) // 3
        c["ctx_hi"] = rng.choice([0, _log(rng, 1, 2048)])
        c["ctx_lo"] = c["ctx_hi"] // 4
        c["kind"] = rng.choice(["bf16", "e4m3"])
        c["rotary"] = rng.choice([c["d"], c["d"] // 2])
        c["interleaved"] = rng.random() < 0.5
        c["fused"] = rng.random() < 0.5
    elif op == "decode":
        c["B"] = _log(rng, 1, 256)
        hi = max(2, min(131072, 300_000 * 1024 // row // c["B"]))
        c["ctx_hi"] = _log(rng, 1, hi)
        c["ctx_lo"] = max(1, c["ctx_hi"] // rng.choice([1, 2, 8, 64]))
        c["kind"] = rng.choice(["bf16", "e4m3"])
    else:
        c["B"] = _log(rng, 1, 16)
        most = 2_000_000_000 // (c["B"] * c["H_q"])  # scores of one head that the plain form holds
        c["new_hi"] = _log(rng, 1, min(4096, int(math.sqrt(most))))
        c["new_lo"] = 1 + (c["new_hi"] - 1) // rng.choice([1, 4])
        room = min(32768, most // c["new_hi"]) - c["new_hi"]
        c["ctx_hi"] = 0 if room < 2 or rng.random() < 0.3 else _log(rng, 1, room)
        c["ctx_lo"] = c["ctx_hi"] // 2
        c["causal"] = rng.random() < 0.8
    return c


def _lengths(case):
    """New tokens and total length of each sequence: the same for every seed."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_lo" in case else 1 for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    # the range of a decoding step is that of whole lengths
    total = ctx if case["op"] == "decode" else [n + c for n, c in zip(new, ctx)]
    return new, total


def _inputs(case, seed):
    """Everything on the GPU that a call takes, from the seed alone."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    new, total = _lengths(case)
    B, H_q, H_kv, d, page = (case[x] for x in ("B", "H_q", "H_kv", "d", "page"))
    width = max(1, -(-max(total) // page))
    pages = sum(-(-n // page) for n in total) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32)
    at = 0
    for b, n in enumerate(total):
        m = -(-n // page)
        table[b, :m] = torch.arange(at, at + m, dtype=torch.int32)
        at += m
    s = dict(case=case, table=order[table.to(dev).long()].contiguous(), lens=torch.tensor(total, dtype=torch.int32, device=dev))
    quant = case.get("kind") == "e4m3"
    s["k"], s["v"] = normal(pages, H_kv, page, d), normal(pages, H_kv, page, d)
    s["k_scale"] = s["v_scale"] = None
    if quant:  # scales that use a good part of e4m3's range
        s["k_scale"] = 0.01 + 0.01 * torch.rand(H_kv, generator=g, device=dev)
        s["v_scale"] = 0.01 + 0.01 * torch.rand(H_kv, generator=g, device=dev)
        s["k"] = (s["k"] * 64).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["v"] = (s["v"] * 64).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    T = sum(new)
    if case["op"] == "append":
        if case["fused"]:  # views of one projection's output
            x = normal(T, H_q + 2 * H_kv, d)
            s["q"], s["new_k"], s["new_v"] = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        else:
            s["q"], s["new_k"], s["new_v"] = normal(T, H_q, d), normal(T, H_kv, d), normal(T, H_kv, d)
        half = case["rotary"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(dev)
    else:
        s["q"] = normal(T, H_q, d)
    s["cu"] = None
    if "new_lo" in case and (case["op"] == "chunk" or case["new_hi"] > 1):
        s["cu"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=dev)
    s["most_new"] = max(new)  # a program that packs its batch knows its longest piece
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from exact_attention_15_gb300 import binding
        s["cache"] = binding.PagedCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        from exact_attention_15_gb300 import binding
        if op == "append":
            q = binding.paged_append(s["cache"], s["q"], s["new_k"], s["new_v"], s["table"], s["lens"], cu_seqlens=s["cu"],
                                     inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
            return {"q": q, "k": s["k"], "v": s["v"]}
        if op == "decode":
            o, lse = binding.paged_decode(s["cache"], s["q"], s["table"], s["lens"])
        else:
            o, lse = binding.paged_forward(s["cache"], s["q"], s["table"], s["lens"], s["cu"], causal=s["case"]["causal"])
        return {"o": o, "lse": lse}
    return {"append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[op](s)


# ------------------------------------------------------------------ plain forms

def _where_new(s):
    """Sequence, place in its chunk and position of every new token."""
    T, B, dev = s["q"].shape[0], s["case"]["B"], s["q"].device
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(B + 1, device=dev)
    t = torch.arange(T, device=dev)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    place = t - cu[seq]
    pos = s["lens"].long()[seq] - (cu[seq + 1] - cu[seq]) + place
    return cu, seq, place, pos


def _rotated(x, pos, inv_freq, interleaved):
    x = x.float()
    angle = pos.double()[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    half = inv_freq.shape[0]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _stored(x, scale, cache):
    if scale is None:
        return x.to(cache.dtype)
    return (x / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)


def _put(cache, page, row, x):
    as_int = torch.uint8 if cache.element_size() == 1 else torch.int16
    cache.view(as_int)[page, :, row] = x.view(as_int)


def _plain_append(s):
    _, seq, _, pos = _where_new(s)
    size, inter = s["case"]["page"], s["case"]["interleaved"]
    page, row = s["table"].long()[seq, pos // size], pos % size
    q = _rotated(s["q"], pos, s["inv_freq"], inter).to(torch.bfloat16)
    _put(s["k"], page, row, _stored(_rotated(s["new_k"], pos, s["inv_freq"], inter), s["k_scale"], s["k"]))
    _put(s["v"], page, row, _stored(s["new_v"].float(), s["v_scale"], s["v"]))
    return {"q": q, "k": s["k"], "v": s["v"]}


def _gathered(cache, scale, table):
    """The sequences' keys or values, [B, H_kv, L, d] in fp32."""
    as_int = torch.uint8 if cache.element_size() == 1 else torch.int16
    x = cache.view(as_int)[table.long()].view(cache.dtype).float()  # [B, width, H_kv, page, d]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _softmax_product(scores, hidden, values):
    """Output and log-sum-exp of the scores that are not hidden; rows without any give 0 and -inf."""
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, values) / torch.where(total == 0, torch.ones_like(total), total)
    return o, (top + total.log()).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    k, v = _gathered(s["k"], s["k_scale"], s["table"]), _gathered(s["v"], s["v_scale"], s["table"])
    past = torch.arange(k.shape[2], device=k.device)[None, :] >= s["lens"][:, None]
    scores = torch.matmul(s["q"].float().view(B, H_kv, H_q // H_kv, d), k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    o, lse = _softmax_product(scores, past[:, None, None, :], v)
    return {"o": o.reshape(B, H_q, d).to(torch.bfloat16), "lse": lse.reshape(B, H_q)}


def _plain_chunk(s):
    c = s["case"]
    B, H_q, H_kv, d = c["B"], c["H_q"], c["H_kv"], c["d"]
    n, group = s["most_new"], H_q // H_kv
    cu, seq, place, _ = _where_new(s)
    rows = (cu[:-1, None] + torch.arange(n, device=cu.device)).clamp_(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, H_kv, group, d).permute(0, 2, 3, 1, 4).reshape(B, H_kv, group * n, d)
    k, v = _gathered(s["k"], s["k_scale"], s["table"]), _gathered(s["v"], s["v_scale"], s["table"])
    key = torch.arange(k.shape[2], device=k.device)
    last = s["lens"].long()[:, None] - 1  # the last key that each new token sees
    if c["causal"]:
        last = last - (cu[1:] - cu[:-1])[:, None] + 1 + torch.arange(n, device=k.device)
    hidden = (key[None, None, :] > last[:, :, None]).expand(B, n, key.numel())
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(B, H_kv, group, n, -1)
    o, lse = _softmax_product(scores, hidden[:, None, None], v[:, :, None])
    o = o.reshape(B, H_q, n, d)[seq, :, place]
    return {"o": o.to(torch.bfloat16), "lse": lse.reshape(B, H_q, n)[seq, :, place].t().contiguous()}


# ------------------------------------------------------------------ definition in 64 bits

def exact(case, seed):
    """One sequence at a time, in 64 bits."""
    s = _inputs(case, seed)
    new, total = _lengths(case)
    page, d, group = case["page"], case["d"], case["H_q"] // case["H_kv"]
    if case["op"] == "append":
        freq, pairs = s["inv_freq"], case["rotary"] // 2
        if case["interleaved"]:
            i0 = torch.arange(0, 2 * pairs, 2, device="cuda")
            i1 = i0 + 1
        else:
            i0 = torch.arange(pairs, device="cuda")
            i1 = i0 + pairs
        out = {"q": s["q"].double(), "k": s["k"].double(), "v": s["v"].double()}
        t0 = 0
        for b, n in enumerate(new):
            pos = torch.arange(total[b] - n, total[b], device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None].double() * freq)[:, None, :]
            spots = s["table"][b].long()[pos // page], pos % page
            for name, x in (("q", s["q"]), ("k", s["new_k"]), ("v", s["new_v"])):
                y = x[t0:t0 + n].double()
                if name != "v":
                    z = torch.complex(y[..., i0], y[..., i1]) * turn
                    y[..., i0], y[..., i1] = z.real, z.imag
                if name == "q":
                    out["q"][t0:t0 + n] = y
                    continue
                if s[name + "_scale"] is not None:
                    y = (y / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
                out[name][spots[0], :, spots[1]] = y
            t0 += n
        return out
    o, lse, t0 = [], [], 0
    for b, n in enumerate(new):
        L = total[b]
        ids = s["table"][b, :-(-L // page)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name].view(torch.uint8 if s[name].element_size() == 1 else torch.int16)[ids].view(s[name].dtype).double()
            x = x.transpose(1, 2).reshape(-1, case["H_kv"], d)[:L]
            if s[name + "_scale"] is not None:
                x = x * s[name + "_scale"].double()[:, None]
            kv.append(x.repeat_interleave(group, dim=1).transpose(0, 1))
        q = s["q"][t0:t0 + n].double().transpose(0, 1)
        w = q @ kv[0].transpose(1, 2) / math.sqrt(d)
        if case.get("causal"):
            w += torch.full((n, L), -math.inf, dtype=torch.float64, device="cuda").triu(L - n + 1)
        lse.append(torch.logsumexp(w, -1))
        o.append((torch.softmax(w, -1) @ kv[1]).transpose(0, 1))
        t0 += n
    o = torch.cat(o)
    return {"o": o, "lse": torch.cat(lse, dim=1) if case["op"] == "chunk" else torch.stack(lse).squeeze(-1)}


def work(case):
    new, total = _lengths(case)
    H_q, H_kv, d = case["H_q"], case["H_kv"], case["d"]
    size = 1 if case.get("kind") == "e4m3" else 2
    T, L = sum(new), sum(total)
    if case["op"] == "append":
        read = T * (H_q + 2 * H_kv) * d * 2
        return {"bytes": read + T * H_q * d * 2 + T * 2 * H_kv * d * size, "flops": 3 * T * (H_q + H_kv) * case["rotary"]}
    seen = sum(n * t - (n * (n - 1) // 2 if case.get("causal") else 0) for n, t in zip(new, total))
    # keys and values once, queries once, outputs and log-sum-exp once
    return {"bytes": 2 * L * H_kv * d * size + T * H_q * (4 * d + 4), "flops": 4 * seen * H_q * d}
