"""Cases and plain 64-bit forms for the prompt-side and eviction calls' tests.

Every form is written from its definition, request by request and head by
head, in float64 on the CPU. Slots that hold no token (past a request's
length, and pages no table maps) are filled with NaN and infinities, so a
kernel that lets one of them through shows it.
"""

from __future__ import annotations

import math

import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards

BF16 = 2.0 ** -8    # half a step of bf16, relative
FP32 = 2.0 ** -24   # half a step of fp32, relative


class Batch:
    """Ragged requests over one paged layer: tokens[b] cached, the last news[b] of them new.

    lead, tail: packed rows before the first and behind the last request's."""

    def __init__(self, dev, tokens, news, Hq, Hkv, d, P, seed=0, max_pages=None, lead=0, tail=0,
                 key_scale=1.0):
        self.tokens, self.news, self.Hq, self.Hkv, self.d, self.P = tokens, news, Hq, Hkv, d, P
        self.g, self.B, self.dev = Hq // Hkv, len(tokens), dev
        self.scale = 1.0 / math.sqrt(d)
        gen = torch.Generator().manual_seed(seed)
        self.gen = gen
        pages = [-(-t // P) for t in tokens]
        self.max_pages = max_pages or max(1, max(pages))
        self.n_phys = sum(pages) + 3
        perm = torch.randperm(self.n_phys, generator=gen).to(torch.int32)
        self.table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        shape = (self.n_phys, Hkv, P, d)
        self.k = torch.full(shape, math.nan, dtype=torch.bfloat16)
        self.v = torch.full(shape, math.inf, dtype=torch.bfloat16)
        for b, t in enumerate(tokens):
            k = (torch.randn((t, Hkv, d), generator=gen) * key_scale).to(torch.bfloat16)
            v = torch.randn((t, Hkv, d), generator=gen).to(torch.bfloat16)
            self.put(self.k, b, k)
            self.put(self.v, b, v)
        offs = [lead]
        for n in news:
            offs.append(offs[-1] + n)
        self.offs, self.N = offs, offs[-1] + tail
        self.q = torch.randn((self.N, Hq, d), generator=gen).to(torch.bfloat16)

    def put(self, cache, b, rows, start=0):
        """Rows [n, Hkv, d] into request b's slots from `start` on."""
        for i in range(rows.shape[0]):
            s = start + i
            cache[int(self.table[b, s // self.P]), :, s % self.P] = rows[i]

    def rows(self, cache, b, n=None, table=None):
        """Request b's slots [n, Hkv, d]."""
        n = self.tokens[b] if n is None else n
        table = self.table if table is None else table
        s = torch.arange(n)
        return cache[table[b, s // self.P].long(), :, s % self.P] if n else \
            cache.new_zeros((0, self.Hkv, self.d))

    def to_device(self):
        """PagedKV (guarded caches and summaries), offsets and workspace on the device."""
        self.k_dev = guards.guarded_like(self.k.to(self.dev), "k_cache")
        self.v_dev = guards.guarded_like(self.v.to(self.dev), "v_cache")
        self.summ_dev = guards.guarded((self.B, self.Hkv, self.max_pages, 2, self.d), torch.bfloat16,
                                       self.dev, fill=0, what="summaries")
        self.table_dev = self.table.to(self.dev)
        self.lens_dev = torch.tensor(self.tokens, dtype=torch.int32, device=self.dev)
        self.offs_dev = torch.tensor(self.offs, dtype=torch.int32, device=self.dev)
        self.kv = B.PagedKV(self.k_dev, self.v_dev, self.summ_dev, self.table_dev, self.lens_dev,
                            self.Hq)
        self.ws = guards.guarded_workspace(self.kv)
        return self.kv

    def request_of(self):
        """(request, slot, packed row) of every new token."""
        for b in range(self.B):
            for i in range(self.news[b]):
                yield b, self.tokens[b] - self.news[b] + i, self.offs[b] + i


def logits(batch, b, h, q, valid=None):
    """[g, n, T] scaled logits of head h's group, masked slots -inf, and sum |q_i k_i| * scale."""
    n, T = batch.news[b], batch.tokens[b]
    k = batch.rows(batch.k, b)[:, h].double()
    qg = q[batch.offs[b]:batch.offs[b] + n, h * batch.g:(h + 1) * batch.g].double()
    x = torch.einsum("ngd,td->gnt", qg, k) * batch.scale
    size = torch.einsum("ngd,td->gnt", qg.abs(), k.abs()) * batch.scale
    see = torch.arange(T) <= torch.arange(T - n, T)[:, None]
    if valid is not None:
        see = see & valid[b][None, :T]
    return x.masked_fill(~see, -math.inf), size.masked_fill(~see, 0.0)


def attend(batch, q, valid=None):
    """(out, lse, bound of out's error, bound of lse's error) in float64, rows of no request NaN.

    Bounds: q.k is summed in fp32 (d products), each probability is rounded to
    bf16 once, the output once more; the sums and the exponentials add a few
    fp32 steps a term."""
    out = torch.full((batch.N, batch.Hq, batch.d), math.nan, dtype=torch.float64)
    lse = torch.full((batch.N, batch.Hq), math.nan, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(batch.B):
        n, T = batch.news[b], batch.tokens[b]
        if n == 0:
            continue
        at = slice(batch.offs[b], batch.offs[b] + n)
        for h in range(batch.Hkv):
            heads = slice(h * batch.g, (h + 1) * batch.g)
            x, size = logits(batch, b, h, q, valid)
            v = batch.rows(batch.v, b)[:, h].double()
            if valid is not None:
                v = torch.where(valid[b][:T, None], v, torch.zeros_like(v))
            p = torch.exp(x - torch.logsumexp(x, -1, keepdim=True).clamp(min=-1e300))
            out[at, heads] = torch.einsum("gnt,td->ngd", p, v)
            lse[at, heads] = torch.logsumexp(x, -1).T
            # relative error of each probability
            dx = (batch.d + 4) * FP32 * size.amax(-1).T + 2.0 ** -20 + T * FP32
            ltol[at, heads] = dx + 4 * FP32 * lse[at, heads].abs().nan_to_num(posinf=0.0)
            mass = torch.einsum("gnt,td->ngd", p, v.abs())
            tol[at, heads] = BF16 * out[at, heads].abs() + (BF16 + 2 * dx)[..., None] * mass
    return out, lse, tol * (1 + 2.0 ** -6), ltol


def chunk_weights(batch, q, lse, decay, w_in, valid=None):
    """(w_out, bound) [B, Hkv, slots] in float64; slots past a request's length NaN."""
    slots = batch.max_pages * batch.P
    out = torch.full((batch.B, batch.Hkv, slots), math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(batch.B):
        n, T = batch.news[b], batch.tokens[b]
        for h in range(batch.Hkv):
            w = torch.zeros(T, dtype=torch.float64)
            if w_in is not None:
                w[:T - n] = decay * w_in[b, h, :T - n].double()
            out[b, h, :T], tol[b, h, :T] = w, 2 * FP32 * w
            if n == 0:
                continue
            x, size = logits(batch, b, h, q, valid)
            l = lse[batch.offs[b]:batch.offs[b] + n, h * batch.g:(h + 1) * batch.g].double().T[..., None]
            p = torch.where(torch.isinf(l), torch.zeros_like(x), torch.exp(x - l.nan_to_num(neginf=0.0)))
            dx = (batch.d + 4) * FP32 * size + 4 * FP32 * l.abs().nan_to_num(posinf=0.0) + 2.0 ** -20 \
                + batch.g * n * FP32
            out[b, h, :T] += p.sum((0, 1))
            tol[b, h, :T] += (p * dx).sum((0, 1)) + 2 * FP32 * out[b, h, :T]
    return out, tol


def norm_rotate(batch, qkv, positions, q_weight, k_weight, eps, inv_freq, interleaved):
    """(q, k, v) of the packed rows in float64, and the size of each rotated pair."""
    Hq, Hkv, d = batch.Hq, batch.Hkv, batch.d
    x = qkv.double()

    def one(y, w):
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
        if inv_freq is None:
            return y, y.abs()
        half = inv_freq.numel()
        ang = positions.double()[:, None] * inv_freq.double()
        cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        z, size = y.clone(), y.abs()
        ia = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = y[..., ia], y[..., ib]
        z[..., ia], z[..., ib] = a * cos - b * sin, b * cos + a * sin
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
        return z, size

    q, qs = one(x[:, :Hq], q_weight)
    k, ks = one(x[:, Hq:Hq + Hkv], k_weight)
    return q, qs, k, ks, qkv[:, Hq + Hkv:]


def evict_ids(w, T, keep, recent):
    """Kept slots of one head, ascending: a NaN counts as the largest, ties stay at the lower slot."""
    n = min(T, keep)
    if T <= keep:
        return list(range(T))
    m = T - recent
    key = [math.inf if math.isnan(x) else x for x in w[:m].tolist()]
    nan = [math.isnan(x) for x in w[:m].tolist()]
    order = sorted(range(m), key=lambda i: (not nan[i], -key[i], i))
    return sorted(order[:n - recent] + list(range(m, T)))


def close(got, want, tol, what):
    """got within tol of want wherever want is finite; infinities equal."""
    got, want = got.double().cpu(), want.cpu()
    fin = torch.isfinite(want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    err = (got - want).abs()[fin]
    bad = ~(err <= tol[fin])
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                                 f"{float((err / tol[fin].clamp(min=1e-300)).max()):.3g} of its bound")
