"""asp_chunk_attention against its definition in 64 bits.

Head layouts, page sizes, lengths from one token on, chunks that end inside a
page and inside a key tile, requests without rows, rows of no request,
garbage (NaN, infinity) in every slot that holds no token, logits that rise
along the cache, bad pages and offsets, another stream, graph replays.
"""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R

pytestmark = pytest.mark.gpu


def call(batch, q=None, scale=None, stream=None):
    q = (batch.q if q is None else q).to(batch.dev)
    out = guards.guarded((batch.N, batch.Hq, batch.d), torch.bfloat16, batch.dev, fill=7.0,
                         what="out")
    lse = guards.guarded((batch.N, batch.Hq), torch.float32, batch.dev, fill=7.0, what="lse")
    B.asp_chunk_attention(batch.kv, q, batch.offs_dev, scale or batch.scale, out, lse, batch.ws,
                          stream)
    return out, lse


def check(batch, out, lse, q=None, valid=None):
    want, wl, tol, ltol = R.attend(batch, batch.q if q is None else q, valid)
    R.close(lse, wl, ltol, "lse")
    R.close(out, want, tol, "out")
    mine = torch.zeros(batch.N, dtype=torch.bool)
    for _, _, row in batch.request_of():
        mine[row] = True
    assert bool((out[~mine] == 7.0).all()) and bool((lse[~mine] == 7.0).all())


RAGGED = [
    ([1], [1]),
    ([128, 129, 127], [128, 129, 1]),
    ([300, 0, 17, 256, 64], [37, 0, 0, 256, 1]),
    ([1030, 513], [260, 65]),
]


@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 64, 16), (8, 2, 128, 16), (8, 1, 128, 64),
                                        (4, 4, 64, 32), (2, 1, 128, 32), (16, 2, 64, 64)])
@pytest.mark.parametrize("tokens,news", RAGGED)
def test_shapes(cuda_device, Hq, Hkv, d, P, tokens, news):
    batch = R.Batch(cuda_device, tokens, news, Hq, Hkv, d, P, seed=P + d, lead=2, tail=3)
    batch.to_device()
    out, lse = call(batch)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 7, 40])
def test_few_rows_over_a_long_cache(cuda_device, d, n):
    """The key axis is split over the whole GPU and joined."""
    batch = R.Batch(cuda_device, [5000, 2049], [n, 1], 8, 2, d, 16, seed=n)
    batch.to_device()
    out, lse = call(batch)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, out, lse)
    again, _ = call(batch)
    assert torch.equal(again, out), "the result depends on timing"


@pytest.mark.parametrize("rise", [0.02, 1.0, 40.0])
@pytest.mark.parametrize("down", [False, True])
def test_logits_that_rise_along_the_cache(cuda_device, rise, down):
    """Each key adds `rise` to the logit of the one before: the running maximum moves at every
    tile (or never, when they fall), and the first keys underflow."""
    batch = R.Batch(cuda_device, [700], [150], 4, 2, 64, 16, seed=1, key_scale=0.05)
    steps = torch.arange(700.0)
    steps = steps.flip(0) if down else steps
    k = batch.rows(batch.k, 0).clone()
    k[:, :, 0] = (rise * 8 * steps / 8)[:, None].to(torch.bfloat16)
    batch.put(batch.k, 0, k)
    batch.q[:, :, 0] = 8.0  # scale 1/8: adds rise per key
    batch.to_device()
    out, lse = call(batch)
    check(batch, out, lse)


def test_large_and_equal_logits(cuda_device):
    batch = R.Batch(cuda_device, [400], [64], 4, 2, 128, 16, seed=3, key_scale=100.0)
    batch.to_device()
    out, lse = call(batch)
    check(batch, out, lse)
    batch = R.Batch(cuda_device, [400], [64], 4, 2, 128, 16, seed=3, key_scale=0.0)
    batch.to_device()
    out, lse = call(batch)
    check(batch, out, lse)


def test_very_negative_logits(cuda_device):
    """Every logit of a row far below zero: the maximum, not zero, is the reference point."""
    batch = R.Batch(cuda_device, [260], [40], 4, 2, 64, 16, seed=4, key_scale=0.1)
    k = batch.rows(batch.k, 0).clone()
    k[:, :, 0] = -3000.0
    batch.put(batch.k, 0, k)
    batch.q[:, :, 0] = 50.0
    batch.to_device()
    out, lse = call(batch)
    check(batch, out, lse)


def test_non_finite_garbage_of_later_keys(cuda_device):
    """A NaN or infinite K of a later token does not reach the rows before it."""
    batch = R.Batch(cuda_device, [200], [100], 4, 2, 64, 16, seed=6)
    batch.to_device()
    want, _ = call(batch)
    k = batch.rows(batch.k, 0).clone()
    k[150:] = math.nan
    k[160] = math.inf
    batch.put(batch.k, 0, k)
    batch.k_dev.copy_(batch.k.to(cuda_device))
    got, _ = call(batch)
    assert torch.equal(got[:50], want[:50])
    assert bool(torch.isnan(got[50:]).all())


@pytest.mark.parametrize("P", [16, 64])
def test_bad_pages_are_skipped(cuda_device, P):
    tokens, news = [600, 3 * P], [100, 3 * P]
    batch = R.Batch(cuda_device, tokens, news, 8, 2, 64, P, seed=8)
    valid = [torch.ones(t, dtype=torch.bool) for t in tokens]
    real = batch.table.clone()
    for b, p, val in ((0, 2, -1), (0, 600 // P, batch.n_phys), (1, 0, 1 << 30)):
        batch.table[b, p] = val
        valid[b][p * P:(p + 1) * P] = False
    batch.to_device()
    out, lse = call(batch)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    batch.table = real  # the form reads the tokens and drops the invalid ones
    check(batch, out, lse, valid=valid)
    rows = slice(batch.offs[1], batch.offs[1] + P)  # these rows see the bad page alone
    assert bool((out[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())


def test_bad_offsets_are_refused_on_the_device(cuda_device):
    batch = R.Batch(cuda_device, [40, 20], [40, 20], 8, 2, 64, 16, seed=9)
    batch.to_device()
    for offs in ([0, 41, 61], [0, 30, 20], [-1, 40, 60], [0, 40, 62]):
        batch.offs_dev.copy_(torch.tensor(offs, dtype=torch.int32))
        call(batch)
        assert B.asp_get_device_error(batch.ws) & B.ASP_DEVERR_OFFSET_RANGE
    batch.offs_dev.copy_(torch.tensor([0, 40, 60], dtype=torch.int32))
    batch.lens_dev.copy_(torch.tensor([1 << 20, 20], dtype=torch.int32))
    call(batch)
    assert B.asp_get_device_error(batch.ws) & B.ASP_DEVERR_SEQ_RANGE


def test_no_rows(cuda_device):
    batch = R.Batch(cuda_device, [40], [0], 8, 2, 64, 16)
    batch.to_device()
    out, lse = call(batch)
    assert out.shape[0] == 0 and B.asp_get_device_error(batch.ws) == 0


def test_many_requests(cuda_device):
    tokens = [1 + (i * 37) % 90 for i in range(300)]
    news = [min(t, (i * 5) % 7) for i, t in enumerate(tokens)]
    batch = R.Batch(cuda_device, tokens, news, 4, 2, 64, 16, seed=12)
    batch.to_device()
    out, lse = call(batch)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, out, lse)


def test_more_requests_than_threads(cuda_device):
    """Every thread of the plan holds several requests; most have a row or none."""
    tokens = [1 + (i * 37) % 40 for i in range(1500)]
    news = [min(t, (i * 5) % 3) for i, t in enumerate(tokens)]
    batch = R.Batch(cuda_device, tokens, news, 2, 1, 64, 16, seed=15)
    batch.to_device()
    out, lse = call(batch)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, out, lse)


def test_rows_of_no_request_may_hold_anything(cuda_device):
    """The tiles of rows reach past a request's last row: what lies there does not come in."""
    batch = R.Batch(cuda_device, [90, 61], [37, 5], 8, 2, 64, 16, seed=16, lead=4, tail=9)
    batch.q[:4] = math.nan
    batch.q[-9:] = math.inf
    batch.to_device()
    out, lse = call(batch)
    check(batch, out, lse)


def test_lengths_and_offsets_that_change_between_replays(cuda_device):
    """A captured call follows the device's lengths and offsets, from many rows to none."""
    batch = R.Batch(cuda_device, [900, 300], [200, 100], 8, 2, 64, 16, seed=17)
    batch.to_device()
    q = batch.q.to(cuda_device)
    out = guards.guarded((batch.N, 8, 64), torch.bfloat16, cuda_device, fill=7.0)
    lse = guards.guarded((batch.N, 8), torch.float32, cuda_device, fill=7.0)
    args = (batch.kv, q, batch.offs_dev, batch.scale, out, lse, batch.ws)
    B.asp_chunk_attention(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.asp_chunk_attention(*args)
    for tokens, news in (([900, 300], [200, 100]), ([512, 17], [1, 17]), ([900, 0], [300, 0]),
                         ([5, 300], [0, 0]), ([128, 300], [128, 172])):
        batch.tokens, batch.news = tokens, news
        batch.offs = [0, news[0], news[0] + news[1]]
        batch.lens_dev.copy_(torch.tensor(tokens, dtype=torch.int32))
        batch.offs_dev.copy_(torch.tensor(batch.offs, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert B.asp_get_device_error(batch.ws) == 0
        check(batch, out, lse)


def test_another_stream_and_graphs_that_share_a_workspace(cuda_device):
    """Two graphs over one workspace, replayed in turn on a stream of their own."""
    a = R.Batch(cuda_device, [3000], [5], 8, 2, 128, 16, seed=13)
    c = R.Batch(cuda_device, [700, 900], [200, 130], 8, 2, 128, 16, seed=14, max_pages=a.max_pages)
    for x in (a, c):
        x.to_device()
    ws = max((a.ws, c.ws), key=lambda t: t.numel())
    a.ws = c.ws = ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in (a, c):
            call(x, stream=side)
            outs.append(call(x, stream=side))
    side.synchronize()
    for x, (out, lse) in zip((a, c), outs):
        q = x.q.to(cuda_device)
        x.keep = q
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.asp_chunk_attention(x.kv, q, x.offs_dev, x.scale, out, lse, ws)
        graphs.append(g)
    for out, lse in outs:
        out.fill_(7.0)
        lse.fill_(7.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            for g in graphs:
                g.replay()
    side.synchronize()
    assert B.asp_get_device_error(ws) == 0
    for x, (out, lse) in zip((a, c), outs):
        check(x, out, lse)


@pytest.mark.parametrize("Hq,Hkv,d,P", [(2, 1, 64, 16), (8, 2, 128, 16), (4, 4, 128, 64), (8, 1, 64, 32)])
@pytest.mark.parametrize("tokens,news", [
    ([4099], [3]),               # a split item whose rows end inside a warp
    ([131, 77], [131, 77]),      # whole items that do, over a last tile with empty slots
    ([2051, 1500], [37, 291])])  # both
def test_rows_that_end_inside_a_warp(cuda_device, Hq, Hkv, d, P, tokens, news):
    """Some lanes of a warp have a row, a key or a place to write, and others have none."""
    batch = R.Batch(cuda_device, tokens, news, Hq, Hkv, d, P, seed=sum(news), lead=1, tail=2)
    batch.to_device()
    out, lse = call(batch)
    for _ in range(3):
        again, lse_again = call(batch)
        assert torch.equal(again, out) and torch.equal(lse_again, lse)
    assert B.asp_get_device_error(batch.ws) == 0
    check(batch, out, lse)
