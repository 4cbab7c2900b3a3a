"""The prompt-side and eviction operators of the paged cache, as they are measured.

Five operators work on one layer's paged K/V cache: the norm, rotation and
write of new tokens ("append"), the attention of a chunk of new tokens over
the cache ("attend"), the attention weight that every cached token receives
from a chunk ("weigh_chunk") or from one decoded token per request over its
page lists ("weigh_decode"), and the eviction of the tokens with the least
weight ("evict"). `run` computes them in plain torch, or, where `own` is true,
through the package's calls.
"""

import math

import numpy as np
import torch

own = False

EPS = 1e-6
ROPE_BASE = 500000.0
DECAY = 0.98  # of the weight accumulated before this call


def _case(name, op, batch, heads, kv_heads, dim, page, context, new, **more):
    """context: tokens of the longest request, the new ones counted; new: its new tokens."""
    c = dict(name=name, op=op, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
             context=context, new=new)
    c.update(more)
    return c


def listed():
    return [
        # one decoded token of each of 64 requests: the smallest step a server makes, often
        _case("append_decode64", "append", 64, 32, 8, 128, 16, 2049, 1, fp32_q=True),
        # eight ragged prompts packed into one prefill batch, about 16k tokens
        _case("append_prompts", "append", 8, 32, 8, 128, 16, 3001, 2731, fp32_q=False),
        # a short follow-up in a small model's conversation: latency counts
        _case("attend_tiny", "attend", 1, 8, 2, 64, 16, 2048, 33),
        # whole prompts from an empty cache, ragged
        _case("attend_prompts8k", "attend", 2, 32, 8, 128, 16, 8192, 8192),
        # one chunk of a chunked prefill deep inside a long prompt
        _case("attend_chunk32k", "attend", 1, 32, 8, 128, 16, 32768, 2048),
        # a few drafted tokens a request checked against long contexts (wide group, large pages)
        _case("attend_verify64k", "attend", 8, 64, 8, 128, 64, 65536, 5),
        # the weights of a short ragged chunk, small heads
        _case("weigh_chunk2k", "weigh_chunk", 4, 8, 2, 64, 16, 2048, 257),
        # the weights that the last chunk of a long prompt gives its cache, before an eviction
        _case("weigh_chunk32k", "weigh_chunk", 1, 32, 8, 128, 16, 32768, 2048),
        # a decode step's weights over all pages of middling ragged contexts
        _case("weigh_decode4k", "weigh_decode", 8, 32, 8, 128, 16, 4099, 1, share=1.0),
        # a decode step's weights over the 30% of pages that a selection kept, at 128k
        _case("weigh_decode128k", "weigh_decode", 4, 32, 8, 128, 16, 131072, 1, share=0.3),
        # a small cache cut to half
        _case("evict_2k", "evict", 1, 8, 2, 64, 16, 2048, 1, keep=1024, recent=128),
        # eight prompts of 32k cut to half before they are decoded
        _case("evict_32k", "evict", 8, 32, 8, 128, 16, 32768, 1, keep=16384, recent=1024),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["append", "append", "attend", "attend", "attend", "weigh_chunk", "weigh_decode",
                     "evict"])
    heads, kv_heads = rng.choice([(8, 2), (32, 8), (64, 8), (8, 8), (16, 4), (4, 1)])
    dim, page = rng.choice([64, 128]), rng.choice([16, 16, 32, 64])
    if op == "append":
        batch = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log_int(rng, 2, max(2, 10000 // batch))
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    context=new + _log_int(rng, 1, 2000), new=new, fp32_q=rng.random() < 0.5)
    if op in ("attend", "weigh_chunk"):
        context = _log_int(rng, 100, 32768)
        new = _log_int(rng, 1, min(context, 4000))
        # padded scores of the plain form: at most those of the largest listed case
        batch = max(1, min(_log_int(rng, 1, 8), int(2e9 / (context * new * heads))))
        return dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                    context=context, new=new)
    if op == "weigh_decode":
        context = _log_int(rng, 50, 65536)
        return dict(op=op, batch=_log_int(rng, 1, min(32, max(1, 260000 // context))), heads=heads,
                    kv_heads=kv_heads, dim=dim, page=page, context=context, new=1,
                    share=rng.choice([1.0, 0.1, 0.3, 0.6]))
    context = _log_int(rng, 300, 40000)
    keep = rng.randrange(context // 8, context)
    return dict(op=op, batch=_log_int(rng, 1, min(16, max(1, 260000 // context))), heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, context=context, new=1, keep=keep,
                recent=rng.randrange(0, keep // 2))


def _lengths(case):
    """Tokens and new tokens of each request: the first is the longest, the others ragged."""
    b, t, n = case["batch"], case["context"], case["new"]
    fr = [1.0 - 0.45 * ((i * 0.6180339887) % 1.0) for i in range(b)]
    news = [max(1, int(n * f)) for f in fr]
    if t == n:
        return news, news
    return [max(k, int(t * f)) for k, f in zip(news, fr)], news


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    op, B, Hq, Hkv = case["op"], case["batch"], case["heads"], case["kv_heads"]
    d, P = case["dim"], case["page"]
    tokens, news = _lengths(case)
    max_pages = -(-max(tokens) // P)
    n_pages = [-(-t // P) for t in tokens]
    extra = [-(-min(t, case["keep"]) // P) for t in tokens] if op == "evict" else [0] * B
    n_phys = sum(n_pages) + sum(extra) + 4
    perm = torch.randperm(n_phys, generator=cpu).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    dst = torch.full((B, max_pages), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :n_pages[b]] = perm[at:at + n_pages[b]]
        at += n_pages[b]
    for b in range(B):
        dst[b, :extra[b]] = perm[at:at + extra[b]]
        at += extra[b]
    offs = [0]
    for n in news:
        offs.append(offs[-1] + n)
    N = offs[-1]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    s = dict(case=case, N=N, table=table.to(dev), dst=dst.to(dev), tokens=ints(tokens),
             offsets=ints(offs), max_new=max(news), max_pages=max_pages, scale=1.0 / math.sqrt(d))
    # where each new token goes: its request and its slot
    req = torch.repeat_interleave(torch.arange(B), torch.tensor(news))
    first = torch.tensor([t - n for t, n in zip(tokens, news)])
    slot = torch.arange(N) - torch.tensor(offs)[req] + first[req]
    s["req"], s["slot"] = req.to(dev), slot.to(dev)
    s["k"], s["v"] = normal(n_phys, Hkv, P, d), normal(n_phys, Hkv, P, d)
    s["summaries"] = torch.zeros((B, Hkv, max_pages, 2, d), dtype=torch.bfloat16, device=dev)
    if op == "append":
        s["qkv"] = normal(N, Hq + 2 * Hkv, d)
        s["q_weight"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(torch.bfloat16)
        s["k_weight"] = (1 + 0.2 * normal(d, dtype=torch.float32)).to(torch.bfloat16)
        s["inv_freq"] = (ROPE_BASE ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).to(
            torch.float32).to(dev)
        # a decoded token's position is far past its slot once a cache was cut back
        shift = 100000 if case["new"] == 1 else 0
        s["positions"] = (slot + shift).to(torch.int32).to(dev)
        s["out"] = torch.empty((N, Hq, d), device=dev,
                               dtype=torch.float32 if case["fp32_q"] else torch.bfloat16)
        _first_summaries(s)
    elif op in ("attend", "weigh_chunk"):
        s["q"] = (1.5 * normal(N, Hq, d, dtype=torch.float32)).to(torch.bfloat16)
        s["out"] = torch.empty((N, Hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((N, Hq), dtype=torch.float32, device=dev)
    elif op == "weigh_decode":
        s["q"] = 1.5 * normal(B, Hq, d, dtype=torch.float32)
        s["lists"], s["lens"] = None, None
        if case["share"] < 1:
            pages = torch.arange(max_pages, device=dev)
            u = torch.rand((B, Hkv, max_pages), generator=g, device=dev)
            have = pages < ints(n_pages)[:, None, None]
            # the newest page is always among those selected
            u = torch.where(pages == ints(n_pages)[:, None, None] - 1, torch.zeros_like(u), u)
            chosen = (u < case["share"]) & have
            key = torch.where(chosen, pages, torch.full_like(pages, max_pages))
            s["lists"] = key.sort(-1).values.clamp(max=max_pages - 1).to(torch.int32)
            s["lens"] = chosen.sum(-1).to(torch.int32)
    if op in ("weigh_chunk", "weigh_decode", "evict"):
        w = torch.rand((B, Hkv, max_pages * P), generator=g, device=dev)
        s["w_in"] = w * w * w * w * 8  # a few heavy tokens, many light ones
        s["w_out"] = torch.zeros_like(s["w_in"])
    if op in ("weigh_chunk", "weigh_decode"):
        s["lse"] = _lse(s)
    if op == "evict":
        s["kept"] = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    if own:
        from adaptive_sparse_paged_gb300 import binding
        s["kv"] = binding.PagedKV(s["k"], s["v"], s["summaries"], s["table"], s["tokens"], Hq)
        s["ws"] = binding.new_workspace(s["kv"])
        s["binding"] = binding
    return s


# ------------------------------------------------------------ the plain forms
def _rows(s, cache):
    """The cache in logical order, padded: 32 bits [B, Hkv, max_pages * P, d]."""
    x = cache[s["table"].clamp(min=0).long()].float()
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _slots(s):
    return torch.arange(s["max_pages"] * s["case"]["page"], device=s["k"].device)


def _first_summaries(s):
    """Channel minimum and maximum of every page's tokens before the new ones."""
    case, Hkv = s["case"], s["case"]["kv_heads"]
    news = s["offsets"][1:] - s["offsets"][:-1]
    keys = _rows(s, s["k"])
    seen = (_slots(s) < (s["tokens"] - news)[:, None])[:, None, :, None]
    shape = (case["batch"], Hkv, s["max_pages"], case["page"], case["dim"])
    lo = keys.masked_fill(~seen, math.inf).view(shape).amin(3)
    hi = keys.masked_fill(~seen, -math.inf).view(shape).amax(3)
    full = torch.stack([lo, hi], 3)
    s["summaries"].copy_(torch.where(torch.isfinite(full), full, torch.zeros_like(full)))


def _append(s):
    case, Hq, Hkv, d = s["case"], s["case"]["heads"], s["case"]["kv_heads"], s["case"]["dim"]
    P = case["page"]
    x = s["qkv"].float()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], s["qkv"][:, Hq + Hkv:]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(y, weight):
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
        a, b = y[..., :d // 2], y[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    q, k = turned(q, s["q_weight"]).to(s["out"].dtype), turned(k, s["k_weight"]).to(torch.bfloat16)
    page = s["slot"] // P
    phys = s["table"][s["req"], page].long()
    s["k"][phys, :, s["slot"] % P] = k
    s["v"][phys, :, s["slot"] % P] = v
    # the pages with new tokens, summarised over all their tokens
    pages = s["k"][phys].float()
    valid = (page * P)[:, None] + torch.arange(P, device=x.device) < s["tokens"][s["req"], None]
    valid = valid[:, None, :, None]
    lo = pages.masked_fill(~valid, math.inf).amin(2)
    hi = pages.masked_fill(~valid, -math.inf).amax(2)
    s["summaries"][s["req"], :, page] = torch.stack([lo, hi], 2).to(torch.bfloat16)
    return dict(q=q, k=s["k"], v=s["v"], summaries=s["summaries"])


def _padded(s, x):
    """Packed rows [N, ...] by request: [B, max_new, ...], and which of them are there."""
    i = torch.arange(s["max_new"], device=x.device)
    at = s["offsets"][:-1, None].long() + i
    there = at < s["offsets"][1:, None]
    return x[at.clamp(max=s["N"] - 1)], there, at


def _logits(s):
    """Scaled, masked products [B, Hkv, g, max_new, slots] of packed queries with all keys."""
    case = s["case"]
    B, Hq, Hkv = case["batch"], case["heads"], case["kv_heads"]
    q, there, at = _padded(s, s["q"].float())
    q = q.view(B, s["max_new"], Hkv, Hq // Hkv, case["dim"]).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.flatten(2, 3), _rows(s, s["k"]).transpose(-1, -2)) * s["scale"]
    x = x.view(B, Hkv, Hq // Hkv, s["max_new"], -1)
    news = (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    pos = (s["tokens"][:, None] - news + torch.arange(s["max_new"], device=x.device))
    seen = (_slots(s) <= pos[..., None]) & there[..., None]
    return x.masked_fill_(~seen[:, None, None], -math.inf), there, at


def _attend(s):
    case = s["case"]
    x, there, at = _logits(s)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), _rows(s, s["v"])).view(*x.shape[:-1], case["dim"])
    o = (o / total).permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    return dict(out=o[there].to(torch.bfloat16), lse=lse[there])


def _before(s, w):
    """The weight that came in: the new tokens had none, and slots past the last stay as they are."""
    news = s["offsets"][1:] - s["offsets"][:-1]
    old = (_slots(s) < (s["tokens"] - news)[:, None])[:, None]
    return torch.where(old, DECAY * w, torch.zeros_like(w))


def _past(s, w):
    return torch.where((_slots(s) < s["tokens"][:, None])[:, None], w, torch.zeros_like(w))


def _weigh_chunk(s):
    x, there, at = _logits(s)
    case = s["case"]
    lse, _, _ = _padded(s, s["lse"])
    lse = lse.view(case["batch"], s["max_new"], case["kv_heads"], -1).permute(0, 2, 3, 1)
    x = x.sub_(lse[..., None]).exp_()
    return _past(s, _before(s, s["w_in"]) + x.sum((2, 3)))


def _decode_logits(s):
    case = s["case"]
    B, Hq, Hkv, P = case["batch"], case["heads"], case["kv_heads"], case["page"]
    q = s["q"].view(B, Hkv, Hq // Hkv, case["dim"])
    x = torch.matmul(q, _rows(s, s["k"]).transpose(-1, -2)) * s["scale"]
    seen = (_slots(s) < s["tokens"][:, None])[:, None].expand(B, Hkv, -1)
    if s["lists"] is not None:
        picked = torch.zeros((B, Hkv, s["max_pages"] + 1), dtype=torch.bool, device=x.device)
        used = torch.arange(s["max_pages"], device=x.device) < s["lens"][..., None]
        picked.scatter_(2, torch.where(used, s["lists"].long(), s["max_pages"]), True)
        seen = seen & picked[..., :-1].repeat_interleave(P, -1)
    return x.masked_fill_(~seen[:, :, None], -math.inf)


def _weigh_decode(s):
    case = s["case"]
    x = _decode_logits(s) - s["lse"].view(case["batch"], case["kv_heads"], -1, 1)
    return _past(s, _before(s, s["w_in"]) + x.exp().sum(2))


def _lse(s):
    """The log-sum-exp rows that the attention call before a weighing left, in 32 bits."""
    case = s["case"]
    if case["op"] == "weigh_decode":
        return torch.logsumexp(_decode_logits(s).double(), -1).float().reshape(
            case["batch"], case["heads"])
    x, there, at = _logits(s)
    lse = torch.logsumexp(x, -1).permute(0, 3, 1, 2).flatten(2, 3)
    return lse[there].contiguous()


def _evict(s):
    case = s["case"]
    B, Hkv, P, keep, recent = (case[k] for k in ("batch", "kv_heads", "page", "keep", "recent"))
    at, T = _slots(s), s["tokens"][:, None, None]
    # the recent slots first, then by weight; a stable sort leaves ties to the lower slot
    rank = torch.where(at >= T - recent, torch.full_like(s["w_in"], math.inf), s["w_in"])
    rank = torch.where(at >= T, torch.full_like(rank, -1.0), rank)
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    n = s["tokens"].clamp(max=keep)
    there = torch.arange(keep, device=at.device) < n[:, None, None]
    last = s["max_pages"] * P
    kept = torch.where(there, order, torch.full_like(order, last)).sort(-1).values
    there = there.expand(B, Hkv, keep)
    src = kept.clamp(max=last - 1)
    s["kept"].copy_(torch.where(there, kept, torch.full_like(kept, -1)))
    s["new_lens"].copy_(n)
    w = torch.gather(s["w_in"], 2, src)
    s["w_out"].zero_()
    s["w_out"][..., :keep] = torch.where(there, w, torch.zeros_like(w))
    b = torch.arange(B, device=at.device)[:, None, None]
    h = torch.arange(Hkv, device=at.device)[None, :, None]
    old = s["table"][b, src // P].long()
    to = torch.arange(keep, device=at.device).expand(B, Hkv, keep)
    new = s["dst"][b, to // P].long()
    hh = h.expand(B, Hkv, keep)
    for_k, for_v = s["k"][old, hh, src % P], s["v"][old, hh, src % P]
    index = new[there], hh[there], (to % P)[there]
    s["k"][index] = for_k[there]
    s["v"][index] = for_v[there]
    pages = -(-keep // P)
    pad = pages * P - keep
    rows = torch.nn.functional.pad(for_k.float(), (0, 0, 0, pad))
    valid = torch.nn.functional.pad(there, (0, pad))[..., None]
    shape = (B, Hkv, pages, P, case["dim"])
    lo = rows.masked_fill(~valid, math.inf).view(shape).amin(3)
    hi = rows.masked_fill(~valid, -math.inf).view(shape).amax(3)
    both = torch.stack([lo, hi], 3)
    s["summaries"][:, :, :pages] = torch.where(torch.isfinite(both), both, torch.zeros_like(both)).to(
        torch.bfloat16)
    return dict(kept=s["kept"], lens=s["new_lens"], weights=s["w_out"], k=s["k"], v=s["v"],
                summaries=s["summaries"])


def _own(s):
    """The package's calls, as a program makes them."""
    op, b, kv, ws = s["case"]["op"], s["binding"], s["kv"], s["ws"]
    if op == "append":
        b.asp_norm_rotate_append(kv, s["qkv"], s["offsets"], s["positions"], s["q_weight"],
                                 s["k_weight"], EPS, s["inv_freq"], False, s["out"], ws)
        return dict(q=s["out"], k=s["k"], v=s["v"], summaries=s["summaries"])
    if op == "attend":
        b.asp_chunk_attention(kv, s["q"], s["offsets"], s["scale"], s["out"], s["lse"], ws)
        return dict(out=s["out"], lse=s["lse"])
    if op == "weigh_chunk":
        b.asp_chunk_weights(kv, s["q"], s["offsets"], s["lse"], s["scale"], DECAY, s["w_in"],
                            s["w_out"], ws)
        return s["w_out"]
    if op == "weigh_decode":
        b.asp_decode_weights(kv, s["q"], s["lists"], s["lens"], s["lse"], s["scale"], DECAY,
                             s["w_in"], s["w_out"], ws)
        return s["w_out"]
    b.asp_weight_evict(kv, s["w_in"], s["case"]["keep"], s["case"]["recent"], s["dst"], s["w_out"],
                       s["kept"], s["new_lens"], ws)
    return dict(kept=s["kept"], lens=s["new_lens"], weights=s["w_out"], k=s["k"], v=s["v"],
                summaries=s["summaries"])


def run(state):
    if own:
        return _own(state)
    return dict(append=_append, attend=_attend, weigh_chunk=_weigh_chunk, weigh_decode=_weigh_decode,
                evict=_evict)[state["case"]["op"]](state)


# ------------------------------------------------------------------ the floors
def work(case):
    """Bytes with every input read once and every output written once, and the products."""
    op, Hq, Hkv, d, P = (case[k] for k in ("op", "heads", "kv_heads", "dim", "page"))
    tokens, news = _lengths(case)
    N, T = sum(news), sum(tokens)
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(tokens, news))
    if op == "append":
        pages = sum(-(-t // P) - (t - n) // P for t, n in zip(tokens, news))
        q_bytes = 4 if case["fp32_q"] else 2
        return dict(bytes=N * d * (2 * (Hq + 2 * Hkv) + q_bytes * Hq + 4 * Hkv) + pages * Hkv * d * 4,
                    flops=N * (Hq + Hkv) * d * 8)
    if op == "attend":
        return dict(bytes=N * Hq * (4 * d + 4) + T * Hkv * d * 4, flops=4 * d * Hq * pairs)
    if op == "weigh_chunk":
        return dict(bytes=N * Hq * (2 * d + 4) + T * Hkv * (2 * d + 8), flops=2 * d * Hq * pairs)
    if op == "weigh_decode":
        seen = T * case["share"]
        return dict(bytes=int(case["batch"] * Hq * (4 * d + 4) + seen * Hkv * 2 * d + T * Hkv * 8),
                    flops=int(2 * d * Hq * seen))
    kept = sum(min(t, case["keep"]) for t in tokens)
    pages = sum(-(-min(t, case["keep"]) // P) for t in tokens)
    return dict(bytes=Hkv * (T * 4 + kept * (8 * d + 8) + pages * 4 * d), flops=0)


# --------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """What `run` returns, request by request and head by head, in 64 bits."""
    s = prepare(case, seed)
    op, B, Hq, Hkv = case["op"], case["batch"], case["heads"], case["kv_heads"]
    d, P = case["dim"], case["page"]
    group = Hq // Hkv
    tokens, news = _lengths(case)
    table = s["table"].cpu().numpy().astype(np.int64)

    def head_rows(cache, b, h, tab=table):
        n = -(-tokens[b] // P)
        idx = torch.from_numpy(tab[b, :n]).to(cache.device)
        return cache[idx, h].reshape(n * P, d)[:tokens[b]]

    if op == "append":
        Kc, Vc, summ = s["k"].double(), s["v"], s["summaries"].double()
        qs = torch.zeros((s["N"], Hq, d), dtype=torch.float64, device=Kc.device)
        row = 0
        for b in range(B):
            n, x = news[b], s["qkv"][row:row + news[b]].double()
            turn = torch.exp(1j * (s["positions"][row:row + n].double()[:, None] *
                                   s["inv_freq"].double()))[:, None]

            def head(y, w):
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * w.double()
                z = torch.complex(y[..., :d // 2], y[..., d // 2:]) * turn
                return torch.cat([z.real, z.imag], -1)

            qs[row:row + n] = head(x[:, :Hq], s["q_weight"])
            keys, vals = head(x[:, Hq:Hq + Hkv], s["k_weight"]), s["qkv"][row:row + n, Hq + Hkv:]
            start = tokens[b] - n
            for p in range(start // P, -(-tokens[b] // P)):
                lo, hi = max(start, p * P), min(tokens[b], (p + 1) * P)
                ph = int(table[b, p])
                Kc[ph, :, lo - p * P:hi - p * P] = keys[lo - start:hi - start].transpose(0, 1)
                Vc[ph, :, lo - p * P:hi - p * P] = vals[lo - start:hi - start].transpose(0, 1)
                page = Kc[ph, :, :hi - p * P]
                summ[b, :, p, 0], summ[b, :, p, 1] = page.amin(1), page.amax(1)
            row += n
        return dict(q=qs, k=Kc, v=Vc.double(), summaries=summ)
    if op == "evict":
        kept = torch.full((B, Hkv, case["keep"]), -1, dtype=torch.int32)
        weights = torch.zeros_like(s["w_in"], dtype=torch.float64)
        Kc, Vc = s["k"].clone(), s["v"].clone()
        summ = s["summaries"].clone()
        new = s["dst"].cpu().numpy().astype(np.int64)
        all_w = s["w_in"].cpu().numpy().astype(np.float64)
        for b in range(B):
            n = min(tokens[b], case["keep"])
            safe = tokens[b] - min(case["recent"], tokens[b])
            for h in range(Hkv):
                w = all_w[b, h, :tokens[b]]
                if n < tokens[b]:
                    by_weight = np.lexsort((np.arange(safe), -w[:safe]))
                    ids = np.sort(np.concatenate([by_weight[:n - case["recent"]],
                                                  np.arange(safe, tokens[b])]))
                else:
                    ids = np.arange(n)
                kept[b, h, :n] = torch.from_numpy(ids.astype(np.int32))
                ids = torch.from_numpy(ids).to(Kc.device)
                weights[b, h, :n] = s["w_in"][b, h][ids].double()
                i = torch.arange(n, device=Kc.device)
                pages = torch.from_numpy(new[b]).to(Kc.device)[i // P]
                keys = head_rows(s["k"], b, h)[ids]
                Kc[pages, h, i % P] = keys
                Vc[pages, h, i % P] = head_rows(s["v"], b, h)[ids]
                full = n // P
                if full:
                    blocks = keys[:full * P].view(full, P, d)
                    summ[b, h, :full, 0], summ[b, h, :full, 1] = blocks.amin(1), blocks.amax(1)
                if n % P:
                    summ[b, h, full, 0] = keys[full * P:].amin(0)
                    summ[b, h, full, 1] = keys[full * P:].amax(0)
        lens = torch.tensor([min(t, case["keep"]) for t in tokens], dtype=torch.int32)
        return dict(kept=kept, lens=lens, weights=weights, k=Kc.double(), v=Vc.double(),
                    summaries=summ.double())
    if op == "attend":
        out = torch.zeros((s["N"], Hq, d), dtype=torch.float64, device=s["k"].device)
        lse = torch.zeros((s["N"], Hq), dtype=torch.float64, device=s["k"].device)
    else:
        out = torch.zeros_like(s["w_in"], dtype=torch.float64)
    row = 0
    for b in range(B):
        n, t = news[b], tokens[b]
        see = torch.arange(t, device=s["k"].device) <= torch.arange(t - n, t, device=s["k"].device)[:, None]
        for h in range(Hkv):
            keys = head_rows(s["k"], b, h).double()
            if op == "weigh_decode" and s["lists"] is not None:
                mine = s["lists"][b, h, :int(s["lens"][b, h])].long()
                listed_page = torch.zeros(-(-t // P), dtype=torch.bool, device=keys.device)
                listed_page[mine] = True
                see = listed_page.repeat_interleave(P)[:t][None]
            if op != "attend":
                out[b, h, :t - n] = DECAY * s["w_in"][b, h, :t - n].double()
            for q_head in range(h * group, (h + 1) * group):
                q = s["q"][row:row + n, q_head].double()
                x = (q @ keys.T) / math.sqrt(d)
                if op == "attend":
                    x = x.masked_fill(~see, -math.inf)
                    lse[row:row + n, q_head] = torch.logsumexp(x, -1)
                    out[row:row + n, q_head] = torch.softmax(x, -1) @ head_rows(s["v"], b, h).double()
                else:
                    p = torch.exp(x - s["lse"][row:row + n, q_head].double()[:, None])
                    out[b, h, :t] += (p * see).sum(0)
        row += n
    return dict(out=out, lse=lse) if op == "attend" else out
