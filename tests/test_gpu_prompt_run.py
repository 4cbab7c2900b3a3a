"""The prompt-side calls, eviction and decoding one after the other, as a server makes them.

Two layers: a chunk of whole prompts, a second chunk, eviction in place, then decode steps
over the cut cache (norm + rotation + append with positions past the slots, selection,
sparse attention, weights). Every stage is checked against its definition in 64 bits on
what the stage before left on the device.
"""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from adaptive_sparse_paged_gb300.step import ChunkStep, DecodeStep, evict
from tests import guards
from tests import prompt_ref as R

pytestmark = pytest.mark.gpu

L, Hq, Hkv, d, P = 2, 8, 2, 64, 16
G = Hq // Hkv
EPS = 1e-6


class Model:
    """Layers' caches with a table of their own; the batch form of one layer for the checks."""

    def __init__(self, dev, max_tokens, seed):
        self.dev = dev
        self.gen = torch.Generator().manual_seed(seed)
        batch = len(max_tokens)
        self.max_pages = -(-max(max_tokens) // P)
        n_phys = batch * self.max_pages + 2
        self.table = torch.randperm(n_phys, generator=self.gen)[:batch * self.max_pages].view(
            batch, self.max_pages).to(torch.int32)
        self.table_dev = self.table.to(dev)
        shape = (n_phys, Hkv, P, d)
        self.k = [guards.guarded(shape, torch.bfloat16, dev, fill=math.nan, what="k") for _ in range(L)]
        self.v = [guards.guarded(shape, torch.bfloat16, dev, fill=math.nan, what="v") for _ in range(L)]
        self.summ = [guards.guarded((batch, Hkv, self.max_pages, 2, d), torch.bfloat16, dev, fill=0)
                     for _ in range(L)]
        self.qw = (1 + 0.3 * torch.randn((L, d), generator=self.gen)).to(torch.bfloat16)
        self.kw = (1 + 0.3 * torch.randn((L, d), generator=self.gen)).to(torch.bfloat16)
        self.freq = (10000.0 ** (-torch.arange(0, d, 2) / d)).float()
        self.batch = batch

    def kvs(self, lens):
        lens_dev = torch.tensor(lens, dtype=torch.int32, device=self.dev)
        return [B.PagedKV(self.k[l], self.v[l], self.summ[l], self.table_dev, lens_dev, Hq)
                for l in range(L)]

    def form(self, l, tokens, news):
        """The layer as prompt_ref sees it, read back from the device."""
        f = R.Batch.__new__(R.Batch)
        f.tokens, f.news, f.Hq, f.Hkv, f.d, f.P, f.g = tokens, news, Hq, Hkv, d, P, G
        f.B, f.scale, f.max_pages, f.table = self.batch, 1.0 / math.sqrt(d), self.max_pages, self.table
        f.k, f.v = self.k[l].cpu(), self.v[l].cpu()
        offs = [0]
        for n in news:
            offs.append(offs[-1] + n)
        f.offs, f.N = offs, offs[-1]
        return f

    def summaries_hold(self, l, tokens):
        f = self.form(l, tokens, [0] * self.batch)
        got = self.summ[l].float().cpu()
        for b, t in enumerate(tokens):
            rows = f.rows(f.k, b).float()
            for p in range(-(-t // P)):
                part = rows[p * P:min(t, (p + 1) * P)]
                assert torch.equal(got[b, :, p, 0], part.amin(0)), (l, b, p)
                assert torch.equal(got[b, :, p, 1], part.amax(0)), (l, b, p)


def chunk(model, tokens, news, weights, w_before, decay, captured):
    dev = model.dev
    N = sum(news)
    qkv = torch.randn((L, N, Hq + 2 * Hkv, d), generator=model.gen).to(torch.bfloat16)
    offs = torch.tensor([0] + list(torch.tensor(news).cumsum(0)), dtype=torch.int32, device=dev)
    step = ChunkStep(model.kvs(tokens), qkv.to(dev), offs, model.freq.to(dev), model.qw.to(dev),
                     model.kw.to(dev), eps=EPS, weights=weights, decay=decay)
    step.run()
    if captured:  # the replay starts from the same weights
        torch.cuda.synchronize()
        first = [t.clone() for t in (step.out, step.lse, weights)]
        step.capture()
        weights.copy_(w_before)
        step.replay()
        torch.cuda.synchronize()
        for x, y in zip(first, (step.out, step.lse, weights)):
            assert torch.equal(x, y)
    assert B.asp_get_device_error(step.ws) == 0
    for l in range(L):
        f = model.form(l, tokens, news)
        pos = torch.cat([torch.arange(t - n, t) for t, n in zip(tokens, news)])
        q, qs, k, ks, v = R.norm_rotate(f, qkv[l], pos, model.qw[l], model.kw[l], EPS, model.freq, False)
        R.close(step.q[l], q, R.BF16 * q.abs() + 2.0 ** -20 * qs, "q")
        for b, slot, row in f.request_of():
            at = int(model.table[b, slot // P]), slice(None), slot % P
            R.close(f.k[at], k[row], R.BF16 * k[row].abs() + 2.0 ** -20 * ks[row], "k")
            assert torch.equal(f.v[at], v[row])
        model.summaries_hold(l, tokens)
        q_dev = step.q[l].cpu()
        out, lse, tol, ltol = R.attend(f, q_dev)
        R.close(step.out[l], out, tol, "out")
        R.close(step.lse[l], lse, ltol, "lse")
        want, wtol = R.chunk_weights(f, q_dev, step.lse[l].cpu(), decay, w_before[l].cpu())
        got = weights[l].cpu()
        for b, t in enumerate(tokens):
            R.close(got[b, :, :t], want[b, :, :t], wtol[b, :, :t], "weights")
    return step


def test_prompt_evict_decode(cuda_device):
    dev = cuda_device
    model = Model(dev, [160, 100], seed=1)
    weights = torch.zeros((L,) + B.weights_shape(model.kvs([1, 1])[0]), device=dev)
    start = weights.clone()
    chunk(model, [70, 33], [70, 33], weights, start, 1.0, captured=False)
    before = weights.clone()
    step = chunk(model, [141, 33], [71, 0], weights, before, 0.9, captured=True)

    # ---- eviction in place
    tokens, keep, recent = [141, 33], 60, 16
    kvs = model.kvs(tokens)
    forms = [model.form(l, tokens, [0, 0]) for l in range(L)]
    w = weights.cpu().clone()
    kept, lens = evict(kvs, weights, keep, recent, step.ws)
    assert B.asp_get_device_error(step.ws) == 0
    assert lens.tolist() == [60, 33]
    for l in range(L):
        now = model.form(l, [60, 33], [0, 0])
        for b, t in enumerate(tokens):
            n = min(t, keep)
            old_k, old_v = forms[l].rows(forms[l].k, b), forms[l].rows(forms[l].v, b)
            new_k, new_v = now.rows(now.k, b), now.rows(now.v, b)
            for h in range(Hkv):
                ids = R.evict_ids(w[l, b, h], t, keep, recent)
                assert kept[l, b, h, :n].tolist() == ids
                assert torch.equal(new_k[:, h], old_k[ids, h]) and torch.equal(new_v[:, h], old_v[ids, h])
                assert torch.equal(weights[l, b, h, :n].cpu(), w[l, b, h][ids])
        model.summaries_hold(l, [60, 33])

    # ---- three decode steps over the cut cache; positions go on from the prompt's
    lens, pos = [60, 33], [141, 33]
    for _ in range(3):
        lens = [t + 1 for t in lens]
        kvs = model.kvs(lens)
        qkv = torch.randn((L, 2, Hq + 2 * Hkv, d), generator=model.gen).to(torch.bfloat16)
        q = torch.zeros((L, 2, Hq, d), device=dev)
        before = weights.clone()
        dec = DecodeStep(kvs, q, 0.95, weights=weights, decay=0.9)
        for l in range(L):
            B.asp_norm_rotate_append(kvs[l], qkv[l].to(dev), None,
                                     torch.tensor(pos, dtype=torch.int32, device=dev),
                                     model.qw[l].to(dev), model.kw[l].to(dev), EPS,
                                     model.freq.to(dev), False, q[l], dec.ws)
        dec.run()
        assert B.asp_get_device_error(dec.ws) == 0
        assert dec.launches_per_step >= L * 4
        for l in range(L):
            f = model.form(l, lens, [1, 1])
            want_q, qs, _, _, _ = R.norm_rotate(f, qkv[l], torch.tensor(pos), model.qw[l], model.kw[l],
                                                EPS, model.freq, False)
            R.close(q[l], want_q, R.FP32 * want_q.abs() + 2.0 ** -20 * qs, "q")
            model.summaries_hold(l, lens)
            from tests.test_gpu_weights import decode_form
            lists, ln = dec.lists[l].cpu(), dec.lens[l].cpu()
            want, tol, lse = decode_form(f, q[l].cpu(), lists, ln, dec.lse[l].cpu(), 0.9,
                                         before[l].cpu())
            assert bool((dec.lse[l].cpu() - lse).abs().max() <= 2e-2)  # the decode's own bound
            for b, t in enumerate(lens):
                R.close(weights[l, b, :, :t].cpu(), want[b, :, :t], tol[b, :, :t], "weights")
        pos = [p + 1 for p in pos]


@pytest.mark.parametrize("dim", [64, 128])
def test_two_streams_at_once(cuda_device, dim):
    """Calls with workspaces of their own on two streams: the same results as one by one."""
    dev = cuda_device
    batch = R.Batch(dev, [1500, 700, 64], [300, 60, 1], 8, 2, dim, 16, seed=31)
    kv = batch.to_device()
    q = batch.q.to(dev)
    qd = torch.randn((3, 8, dim), generator=batch.gen).to(dev)
    other = B.new_workspace(kv)

    def outputs():
        return [torch.zeros((batch.N, 8, dim), dtype=torch.bfloat16, device=dev),
                torch.zeros((batch.N, 8), device=dev), B.new_weights(kv), B.new_weights(kv)]

    def first(o, ws, stream=None):
        B.asp_chunk_attention(kv, q, batch.offs_dev, batch.scale, o[0], o[1], ws, stream)

    def second(o, lse, ws, stream=None):
        B.asp_chunk_weights(kv, q, batch.offs_dev, lse, batch.scale, 1.0, None, o[2], ws, stream)
        B.asp_decode_weights(kv, qd, None, None, lse[:3].contiguous(), batch.scale, 1.0, None, o[3],
                             ws, stream)

    want = outputs()
    first(want, batch.ws)
    second(want, want[1], batch.ws)
    torch.cuda.synchronize()
    lse3 = want[1]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = outputs()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(a):
            first(got, batch.ws)
        with torch.cuda.stream(b):
            second(got, lse3, other)
    torch.cuda.synchronize()
    assert B.asp_get_device_error(batch.ws) == 0 and B.asp_get_device_error(other) == 0
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_shape_checks(cuda_device):
    model = Model(cuda_device, [40, 20], seed=2)
    kvs = model.kvs([40, 20])
    offs = torch.tensor([0, 40, 60], dtype=torch.int32, device=cuda_device)
    good = torch.zeros((L, 60, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device=cuda_device)
    with pytest.raises(ValueError, match="qkv"):
        ChunkStep(kvs, good[:1], offs)
    with pytest.raises(ValueError, match="q_offsets"):
        ChunkStep(kvs, good, offs[:2])
    with pytest.raises(ValueError, match="weights"):
        ChunkStep(kvs, good, offs, weights=torch.zeros((L, 2, Hkv, 5), device=cuda_device))
    with pytest.raises(ValueError, match="at least one layer"):
        evict([], None, 4, 1, None)
    ws = B.new_workspace(kvs[0])
    q = torch.zeros((60, Hq, d), dtype=torch.bfloat16, device=cuda_device)
    lse = torch.zeros((60, Hq), device=cuda_device)
    with pytest.raises(TypeError):
        B.asp_chunk_attention(kvs[0], q.float(), offs, 0.1, q, lse, ws)
    with pytest.raises(ValueError):
        B.asp_chunk_attention(kvs[0], q, offs[:2], 0.1, q, lse, ws)
    with pytest.raises(ValueError):
        B.asp_chunk_attention(kvs[0], q.transpose(0, 1), offs, 0.1, q, lse, ws)
    with pytest.raises(B.AspError):
        B.asp_chunk_attention(kvs[0], q, offs, -1.0, q, lse, ws)
    with pytest.raises(B.AspError):
        B.asp_chunk_attention(kvs[0], q, offs, 0.1, q, lse, ws[:256])
    with pytest.raises(TypeError):
        B.asp_norm_rotate_append(kvs[0], good[0], offs, None, None, None, 1e-6, None, False,
                                 q.half(), ws)


@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_capture_leaves_the_weights_alone(cuda_device, decay):
    """capture() and one replay give what one run() gives, the weights among it."""
    dev = cuda_device
    model = Model(dev, [160, 100], seed=5)
    lens = [150, 77]
    for l in range(L):
        model.k[l].copy_(torch.randn(model.k[l].shape, generator=model.gen))
        model.v[l].copy_(torch.randn(model.v[l].shape, generator=model.gen))
    kvs = model.kvs(lens)
    q = torch.randn((L, 2, Hq, d), generator=model.gen).to(dev)
    new = torch.randn((2, L, 2, Hkv, d), generator=model.gen).to(torch.bfloat16).to(dev)
    ws = B.new_workspace(kvs[0])
    for kv in kvs:
        B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, ws)
    start = torch.rand((L,) + tuple(B.weights_shape(kvs[0])), generator=model.gen).to(dev)
    for b, t in enumerate(lens):
        start[:, b, :, t:] = math.nan  # not read
    weights = guards.guarded_like(start, "weights")
    step = DecodeStep(kvs, q, 0.9, append=(new[0], new[1]), weights=weights, decay=decay)
    step.run()
    want = weights.clone()
    step.run()
    twice = weights.clone()
    weights.copy_(start)
    step.capture()
    torch.cuda.synchronize()
    assert torch.equal(weights.view(torch.int32), start.view(torch.int32)), "capture changed the weights"
    for once in (want, twice):
        step.replay()
        torch.cuda.synchronize()
        assert torch.equal(weights.view(torch.int32), once.view(torch.int32))
    assert B.asp_get_device_error(step.ws) == 0
