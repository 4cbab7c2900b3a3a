"""asp_chunk_weights and asp_decode_weights against their definition in 64 bits."""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R
from tests.test_gpu_chunk_attention import RAGGED

pytestmark = pytest.mark.gpu

FILL = 5.0


def lse_of(batch, q, valid=None):
    return R.attend(batch, q, valid)[1].float()


def check(batch, got, want, tol):
    slots = torch.arange(want.shape[-1])
    past = slots[None] >= torch.tensor(batch.tokens)[:, None]
    past = past[:, None].expand(-1, batch.Hkv, -1)
    assert bool((got.cpu()[past] == FILL).all()), "entries past a request's tokens changed"
    R.close(got.cpu()[~past], want[~past], tol[~past], "weights")


@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 64, 16), (8, 2, 128, 16), (8, 1, 128, 64),
                                        (4, 4, 64, 32), (16, 2, 64, 64)])
@pytest.mark.parametrize("tokens,news", RAGGED)
@pytest.mark.parametrize("decay,before", [(1.0, "same"), (0.5, "other"), (0.0, None)])
def test_chunk(cuda_device, Hq, Hkv, d, P, tokens, news, decay, before):
    batch = R.Batch(cuda_device, tokens, news, Hq, Hkv, d, P, seed=P + d, lead=2, tail=3)
    kv = batch.to_device()
    lse = lse_of(batch, batch.q)
    shape = (batch.B, Hkv, batch.max_pages * P)
    w = guards.guarded(shape, torch.float32, cuda_device, fill=FILL, what="w_out")
    start = torch.rand(shape, generator=batch.gen) * 4
    w_in = None
    if before == "same":
        for b, (t, n) in enumerate(zip(tokens, news)):
            w[b, :, :t - n] = start[b, :, :t - n].to(cuda_device)
            w[b, :, t - n:t] = math.nan  # not read: the chunk's own tokens
        w_in = w
    elif before == "other":
        for b, (t, n) in enumerate(zip(tokens, news)):
            start[b, :, t - n:] = math.nan
        w_in = start.to(cuda_device)
    want, tol = R.chunk_weights(batch, batch.q, lse, decay, None if w_in is None else start)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device),
                        batch.scale, decay, w_in, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)


def test_chunk_weights_sum_to_the_rows(cuda_device):
    """With the attention call's own lse every row gives away one unit."""
    batch = R.Batch(cuda_device, [1000, 333], [129, 333], 8, 2, 128, 16, seed=4)
    kv = batch.to_device()
    q = batch.q.to(cuda_device)
    out = torch.empty_like(q)
    lse = torch.empty((batch.N, 8), device=cuda_device)
    w = B.new_weights(kv)
    B.asp_chunk_attention(kv, q, batch.offs_dev, batch.scale, out, lse, batch.ws)
    B.asp_chunk_weights(kv, q, batch.offs_dev, lse, batch.scale, 1.0, None, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    total = w.double().sum(-1).cpu()
    want = torch.tensor([[129.0 * 4] * 2, [333.0 * 4] * 2], dtype=torch.float64)
    # each probability is off by its logit's rounding, under 2^-13 here
    assert bool(((total - want).abs() <= want * 2.0 ** -13).all())


def test_chunk_no_rows_bad_pages_and_masked_rows(cuda_device):
    P = 16
    batch = R.Batch(cuda_device, [100, 40], [20, 0], 8, 2, 64, P, seed=5)
    lse = lse_of(batch, batch.q)
    lse[3] = -math.inf  # a row that saw nothing
    valid = [torch.ones(t, dtype=torch.bool) for t in batch.tokens]
    real = batch.table.clone()
    batch.table[0, 3] = -7
    valid[0][3 * P:4 * P] = False
    kv = batch.to_device()
    batch.table = real
    start = torch.rand((2, 2, batch.max_pages * P), generator=batch.gen)
    w = guards.guarded(start.shape, torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device),
                        batch.scale, 0.25, start.to(cuda_device), w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    want, tol = R.chunk_weights(batch, batch.q, lse, 0.25, start, valid)
    check(batch, w, want, tol)
    # no new rows at all: the weights only decay
    none = R.Batch(cuda_device, [50], [0], 8, 2, 64, P, seed=6)
    kv = none.to_device()
    w_in = torch.rand((1, 2, none.max_pages * P), generator=none.gen)
    w = guards.guarded(w_in.shape, torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, none.q.to(cuda_device), none.offs_dev,
                        torch.zeros((0, 8), device=cuda_device), none.scale, 0.5,
                        w_in.to(cuda_device), w, none.ws)
    assert B.asp_get_device_error(none.ws) == 0
    assert torch.equal(w[..., :50].cpu(), 0.5 * w_in[..., :50])


def test_chunk_rows_of_no_request_may_hold_anything(cuda_device):
    batch = R.Batch(cuda_device, [90, 300], [37, 5], 8, 2, 64, 16, seed=7, lead=4, tail=9)
    lse = lse_of(batch, batch.q)
    lse[:4], lse[-9:] = math.nan, math.inf
    want, tol = R.chunk_weights(batch, batch.q, lse, 1.0, None)
    batch.q[:4], batch.q[-9:] = math.nan, math.inf
    kv = batch.to_device()
    w = guards.guarded((2, 2, batch.max_pages * 16), torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device),
                        batch.scale, 1.0, None, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)


def test_chunk_more_requests_than_threads(cuda_device):
    tokens = [1 + (i * 37) % 40 for i in range(1200)]
    news = [min(t, (i * 5) % 3) for i, t in enumerate(tokens)]
    batch = R.Batch(cuda_device, tokens, news, 2, 1, 64, 16, seed=8)
    kv = batch.to_device()
    lse = lse_of(batch, batch.q).nan_to_num(0.0)
    start = torch.rand((batch.B, 1, batch.max_pages * 16), generator=batch.gen)
    want, tol = R.chunk_weights(batch, batch.q, lse, 0.5, start)
    w = guards.guarded(start.shape, torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device),
                        batch.scale, 0.5, start.to(cuda_device), w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)


@pytest.mark.parametrize("offs,skipped", [([0, 41, 61], [0, 1]), ([0, 30, 20], [1]),
                                          ([-1, 40, 60], [0]), ([0, 40, 62], [1])])
def test_chunk_a_request_with_bad_offsets_is_skipped(cuda_device, offs, skipped):
    """In place: its weights neither decay nor change, its entries of new tokens are not read."""
    batch = R.Batch(cuda_device, [40, 20], [40, 20], 8, 2, 64, 16, seed=9)
    kv = batch.to_device()
    lse = torch.zeros((batch.N, 8), device=cuda_device)
    w = guards.guarded((2, 2, batch.max_pages * 16), torch.float32, cuda_device, fill=FILL)
    batch.offs_dev.copy_(torch.tensor(offs, dtype=torch.int32))
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse, batch.scale, 0.5, w, w,
                        batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_OFFSET_RANGE
    for b in skipped:
        assert bool((w[b] == FILL).all()), b


def test_chunk_skipped_requests_among_many(cuda_device):
    """Requests with more rows than tokens: the others' weights are what they are without them."""
    tokens = [1 + (i * 37) % 600 for i in range(60)]
    news = [min(t, 1 + (i * 29) % 90) for i, t in enumerate(tokens)]
    batch = R.Batch(cuda_device, tokens, news, 4, 2, 64, 16, seed=19)
    kv = batch.to_device()
    bad = list(range(0, 60, 7))
    lens = torch.tensor(tokens, dtype=torch.int32)
    for b in bad:
        lens[b] = news[b] - 1
    batch.lens_dev.copy_(lens)
    lse = lse_of(batch, batch.q)
    start = torch.rand((batch.B, 2, batch.max_pages * 16), generator=batch.gen)
    want, tol = R.chunk_weights(batch, batch.q, lse, 0.5, start)
    w = guards.guarded(start.shape, torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device),
                        batch.scale, 0.5, start.to(cuda_device), w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_OFFSET_RANGE
    for b, t in enumerate(tokens):
        if b in bad:
            assert bool((w[b] == FILL).all()), b
        else:
            R.close(w[b, :, :t].cpu(), want[b, :, :t], tol[b, :, :t], "weights")


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -40, 2.0 ** 20])
def test_chunk_extreme_scales(cuda_device, scale):
    """Logits that vanish, and logits whose softmax is one key's alone."""
    batch = R.Batch(cuda_device, [300, 131], [70, 131], 8, 2, 64, 16, seed=23)
    batch.scale = scale
    if scale > 1:  # small whole numbers: products and sums are exact, and so is the scale
        batch.q = torch.randint(-2, 3, batch.q.shape, generator=batch.gen).to(torch.bfloat16)
        for b, t in enumerate(batch.tokens):
            batch.put(batch.k, b, torch.randint(-2, 3, (t, 2, 64), generator=batch.gen).to(torch.bfloat16))
    kv = batch.to_device()
    lse = lse_of(batch, batch.q)
    if scale > 1:  # a row's largest logit: exact, where the sum's logarithm is under its last bit
        lse = torch.where(torch.isnan(lse), lse, (lse.double() / scale).round().mul(scale).float())
    want, tol = R.chunk_weights(batch, batch.q, lse, 1.0, None)
    if scale > 1:  # one for each key that has its row's largest logit, nothing for the others
        tol = torch.zeros_like(tol)
    w = guards.guarded((2, 2, batch.max_pages * 16), torch.float32, cuda_device, fill=FILL)
    B.asp_chunk_weights(kv, batch.q.to(cuda_device), batch.offs_dev, lse.to(cuda_device), scale, 1.0,
                        None, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)


# ------------------------------------------------------------------ decode form
def decode_case(dev, tokens, Hq, Hkv, d, P, share, seed):
    news = [min(1, t) for t in tokens]
    batch = R.Batch(dev, tokens, news, Hq, Hkv, d, P, seed=seed)
    q = torch.randn((len(tokens), Hq, d), generator=batch.gen)
    lists = torch.full((batch.B, Hkv, batch.max_pages), -9, dtype=torch.int32)
    lens = torch.zeros((batch.B, Hkv), dtype=torch.int32)
    for b, t in enumerate(tokens):
        n = -(-t // P)
        for h in range(Hkv):
            k = min(n, max(1, int(round(share * n)))) if h or share == 1 else n // 3
            ids = torch.randperm(n, generator=batch.gen)[:k]
            lists[b, h, :k], lens[b, h] = ids.sort().values.to(torch.int32), k
    return batch, q, lists, lens


def decode_form(batch, q, lists, lens, lse, decay, w_in):
    want = torch.full((batch.B, batch.Hkv, batch.max_pages * batch.P), math.nan, dtype=torch.float64)
    tol = torch.zeros_like(want)
    out_lse = torch.full((batch.B, batch.Hq), -math.inf, dtype=torch.float64)
    for b, T in enumerate(batch.tokens):
        for h in range(batch.Hkv):
            if T == 0:
                continue
            see = torch.ones(T, dtype=torch.bool)
            if lists is not None:
                pages = torch.zeros(batch.max_pages, dtype=torch.bool)
                pages[lists[b, h, :int(lens[b, h])].long()] = True
                see = pages.repeat_interleave(batch.P)[:T]
            k = batch.rows(batch.k, b)[:, h].double()
            qg = q[b, h * batch.g:(h + 1) * batch.g].double()
            x = (qg @ k.T * batch.scale).masked_fill(~see, -math.inf)
            size = (qg.abs() @ k.abs().T) * batch.scale
            heads = slice(h * batch.g, (h + 1) * batch.g)
            out_lse[b, heads] = torch.logsumexp(x, -1)
            if lse is None:
                continue
            l = lse[b, heads].double()[:, None]
            p = torch.where(torch.isinf(l), torch.zeros_like(x), torch.exp(x - l.nan_to_num(neginf=0.0)))
            # q enters as two bf16 halves: its remainder is under 2^-16 of it, relative
            dx = ((batch.d + 4) * R.FP32 + 2.0 ** -16) * size + 4 * R.FP32 * l.abs().nan_to_num(posinf=0.0) \
                + 2.0 ** -20
            w = torch.zeros(T, dtype=torch.float64)
            if w_in is not None:
                w[:T - 1] = decay * w_in[b, h, :T - 1].double()
            want[b, h, :T] = w + p.sum(0)
            tol[b, h, :T] = 4 * R.FP32 * want[b, h, :T] + (p * dx).sum(0)
    return want, tol, out_lse.float()


@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 64, 16), (32, 8, 128, 16), (8, 1, 128, 64),
                                        (4, 4, 64, 32), (2, 1, 128, 32)])
@pytest.mark.parametrize("tokens", [[1], [300, 0, 17, 256], [2049, 900, 128]])
@pytest.mark.parametrize("share", [None, 0.3, 1.0])
def test_decode(cuda_device, Hq, Hkv, d, P, tokens, share):
    batch, q, lists, lens = decode_case(cuda_device, tokens, Hq, Hkv, d, P, share or 1.0, seed=d + P)
    if share is None:
        lists = lens = None
    kv = batch.to_device()
    start = torch.rand((batch.B, Hkv, batch.max_pages * P), generator=batch.gen) * 3
    for b, t in enumerate(tokens):
        start[b, :, max(0, t - 1):] = math.nan  # the decoded token's entry is not read
    lse = decode_form(batch, q, lists, lens, None, 0.5, start)[2]
    want, tol, _ = decode_form(batch, q, lists, lens, lse, 0.5, start)
    w = guards.guarded(start.shape, torch.float32, cuda_device, fill=FILL, what="w_out")
    dev = lambda x: None if x is None else x.to(cuda_device)  # noqa: E731
    B.asp_decode_weights(kv, dev(q), dev(lists), dev(lens), dev(lse), batch.scale, 0.5, dev(start),
                         w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)
    # in place, summing
    w2 = guards.guarded_like(torch.where(torch.isnan(start), torch.full_like(start, FILL),
                                         start).to(cuda_device), "w in place")
    w2_start = torch.where(torch.isnan(start), torch.zeros_like(start), start)
    want, tol, _ = decode_form(batch, q, lists, lens, lse, 1.0, w2_start)
    B.asp_decode_weights(kv, dev(q), dev(lists), dev(lens), dev(lse), batch.scale, 1.0, w2, w2,
                         batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w2, want, tol)


def test_decode_after_the_sparse_decode(cuda_device):
    """Selection, decode, weights: each head gives away one unit over its list."""
    batch, q, _, _ = decode_case(cuda_device, [3000, 777], 8, 2, 128, 16, 1.0, seed=21)
    kv = batch.to_device()
    q = q.to(cuda_device)
    lists = torch.zeros((2, 2, batch.max_pages), dtype=torch.int32, device=cuda_device)
    lens = torch.zeros((2, 2), dtype=torch.int32, device=cuda_device)
    out, lse = torch.zeros((2, 8, 128), device=cuda_device), torch.zeros((2, 8), device=cuda_device)
    w = B.new_weights(kv)
    B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    B.asp_coverage_select(kv, q, 0.9, 0, lists, lens, batch.ws)
    B.asp_sparse_decode(kv, q, lists, lens, batch.scale, out, lse, batch.ws)
    B.asp_decode_weights(kv, q, lists, lens, lse, batch.scale, 1.0, None, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    total = w.double().sum(-1).cpu()
    assert bool(((total - 4.0).abs() <= 4 * 2.0 ** -12).all()), total


def test_decode_more_segments_than_threads(cuda_device):
    tokens = [(i * 37) % 60 for i in range(700)]
    batch, q, lists, lens = decode_case(cuda_device, tokens, 4, 2, 64, 16, 0.5, seed=23)
    kv = batch.to_device()
    start = torch.rand((batch.B, 2, batch.max_pages * 16), generator=batch.gen)
    lse = decode_form(batch, q, lists, lens, None, 0.5, start)[2]
    want, tol, _ = decode_form(batch, q, lists, lens, lse, 0.5, start)
    w = guards.guarded(start.shape, torch.float32, cuda_device, fill=FILL)
    dev = cuda_device
    B.asp_decode_weights(kv, q.to(dev), lists.to(dev), lens.to(dev), lse.to(dev), batch.scale, 0.5,
                         start.to(dev), w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, w, want, tol)


def test_decode_bad_lists_and_pages(cuda_device):
    batch, q, lists, lens = decode_case(cuda_device, [100, 60], 8, 2, 64, 16, 1.0, seed=22)
    args = lambda: (batch.kv, q.to(cuda_device), lists.to(cuda_device), lens.to(cuda_device),  # noqa: E731
                    torch.zeros((2, 8), device=cuda_device), batch.scale, 1.0, None,
                    guards.guarded((2, 2, batch.max_pages * 16), torch.float32, cuda_device,
                                   fill=FILL), batch.ws)
    batch.to_device()
    lists[0, 1, 0] = 99
    B.asp_decode_weights(*args())
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_LIST_RANGE
    lists[0, 1, 0] = 0
    lens[1, 1] = 1000
    lists[1, 1] = torch.arange(batch.max_pages)
    B.asp_decode_weights(*args())
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_LEN_RANGE
    lens[1, 1] = 1
    batch.table_dev[0, 0] = -1
    B.asp_decode_weights(*args())
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE


@pytest.mark.parametrize("d,P", [(64, 16), (128, 64)])
def test_decode_keys_that_end_inside_a_warp(cuda_device, d, P):
    """Lanes with a key beside lanes of unlisted pages and of slots past the last token."""
    batch, q, lists, lens = decode_case(cuda_device, [1003, 21, 5 * P + 1], 4, 2, d, P, 0.4, seed=d)
    kv = batch.to_device()
    start = torch.rand((batch.B, 2, batch.max_pages * P), generator=batch.gen)
    dev = cuda_device
    for ls, ln in ((lists, lens), (None, None)):
        lse = decode_form(batch, q, ls, ln, None, 0.5, start)[2]
        want, tol, _ = decode_form(batch, q, ls, ln, lse, 0.5, start)
        first = None
        for _ in range(3):
            w = guards.guarded(start.shape, torch.float32, dev, fill=FILL)
            B.asp_decode_weights(kv, q.to(dev), None if ls is None else ls.to(dev),
                                 None if ln is None else ln.to(dev), lse.to(dev), batch.scale, 0.5,
                                 start.to(dev), w, batch.ws)
            assert first is None or torch.equal(first, w)
            first = w
        assert B.asp_get_device_error(batch.ws) == 0
        check(batch, w, want, tol)
