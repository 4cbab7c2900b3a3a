"""asp_norm_rotate_append against its definition in 64 bits.

q (bf16 or fp32), the written K rows, the copied V rows and the page summaries;
pages that fill, start and end inside a chunk, requests without new tokens,
positions far from the slots, both pairings, partial and no rotation, no norm.
"""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R

pytestmark = pytest.mark.gpu


def inv_freq_of(rot, dev):
    return (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().to(dev)


def run(batch, qkv, positions=None, qw=None, kw=None, eps=1e-6, rot=None, interleaved=False,
        dtype=torch.bfloat16, offsets=True, check=True):
    """One call and its comparison; returns the device outputs."""
    dev, d, Hq, Hkv, P = batch.dev, batch.d, batch.Hq, batch.Hkv, batch.P
    rot = d if rot is None else rot
    # the cache holds the tokens before the chunk; the new slots hold garbage
    for b, slot, _ in batch.request_of():
        batch.k[int(batch.table[b, slot // P]), :, slot % P] = math.nan
        batch.v[int(batch.table[b, slot // P]), :, slot % P] = math.inf
    kv = batch.to_device()
    old = torch.tensor([t - n for t, n in zip(batch.tokens, batch.news)], dtype=torch.int32,
                       device=dev)
    before = B.PagedKV(batch.k_dev, batch.v_dev, batch.summ_dev, batch.table_dev, old, Hq)
    B.asp_page_summarize(before, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    q_out = guards.guarded((batch.N, Hq, d), dtype, dev, fill=7.0, what="q_out")
    freq = inv_freq_of(rot, dev) if rot else None
    args = (kv, qkv.to(dev), batch.offs_dev if offsets else None,
            None if positions is None else positions.to(dev), None if qw is None else qw.to(dev),
            None if kw is None else kw.to(dev), eps, freq, interleaved, q_out, batch.ws)
    for _ in range(2):  # idempotent
        B.asp_norm_rotate_append(*args)
    assert B.asp_get_device_error(batch.ws) == 0
    if not check:
        return q_out
    pos = torch.zeros(batch.N, dtype=torch.int64)
    mine = torch.zeros(batch.N, dtype=torch.bool)
    for b, slot, row in batch.request_of():
        pos[row], mine[row] = slot, True
    if positions is not None:
        pos = positions.long()
    q, qs, k, ks, v = R.norm_rotate(batch, qkv, pos, qw, kw, eps,
                                    None if freq is None else freq.cpu(), interleaved)
    # mean, rsqrt, products and the cosine and sine: under 2^-20 of the pair's size
    half = R.BF16 if dtype == torch.bfloat16 else R.FP32
    R.close(q_out[mine], q[mine], (half * q.abs() + 2.0 ** -20 * qs)[mine], "q")
    assert bool((q_out[~mine] == 7.0).all()), "rows of no request were written"
    k_got, v_got = batch.k_dev.cpu(), batch.v_dev.cpu()
    for b, slot, row in batch.request_of():
        ph = int(batch.table[b, slot // P])
        R.close(k_got[ph, :, slot % P], k[row], R.BF16 * k[row].abs() + 2.0 ** -20 * ks[row], "k")
        assert torch.equal(v_got[ph, :, slot % P], v[row]), "v"
        batch.k[ph, :, slot % P], batch.v[ph, :, slot % P] = k_got[ph, :, slot % P], v[row]
    # nothing else of the caches changed, summaries are those of the written keys
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731
    assert same(k_got, batch.k) and same(v_got, batch.v)
    want = torch.zeros_like(batch.summ_dev).cpu()
    for b, t in enumerate(batch.tokens):
        rows = batch.rows(batch.k, b).float()
        for p in range(-(-t // P)):
            part = rows[p * P:min(t, (p + 1) * P)]
            want[b, :, p, 0], want[b, :, p, 1] = part.amin(0), part.amax(0)
    assert torch.equal(batch.summ_dev.cpu(), want), "summaries"
    return q_out


def make(dev, tokens, news, Hq, Hkv, d, P, seed=0, **kw):
    batch = R.Batch(dev, tokens, news, Hq, Hkv, d, P, seed=seed, **kw)
    qkv = torch.randn((batch.N, Hq + 2 * Hkv, d), generator=batch.gen).to(torch.bfloat16)
    qw, kwt = ((1 + 0.3 * torch.randn(d, generator=batch.gen)).to(torch.bfloat16) for _ in range(2))
    return batch, qkv, qw, kwt


@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 64, 16), (32, 8, 128, 16), (8, 8, 128, 64),
                                        (16, 2, 64, 32), (8, 1, 128, 32), (1, 1, 64, 64)])
@pytest.mark.parametrize("tokens,news", [
    ([1], [1]), ([130, 17, 0, 64], [130, 1, 0, 64]), ([77, 200, 33], [5, 131, 0]),
    ([65, 48, 31], [2, 16, 15])])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(cuda_device, Hq, Hkv, d, P, tokens, news, dtype):
    batch, qkv, qw, kw = make(cuda_device, tokens, news, Hq, Hkv, d, P, seed=d + P, lead=3, tail=2)
    run(batch, qkv, qw=qw, kw=kw, dtype=dtype)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (8, False), (24, True), (64, True),
                                             (32, False), (56, False)])
@pytest.mark.parametrize("norm", ["both", "q", "k", "none"])
def test_rotation_and_norm_forms(cuda_device, d, rot, interleaved, norm):
    batch, qkv, qw, kw = make(cuda_device, [70, 19], [41, 3], 8, 2, d, 16, seed=rot)
    run(batch, qkv, qw=qw if norm in ("both", "q") else None,
        kw=kw if norm in ("both", "k") else None, rot=rot, interleaved=interleaved,
        dtype=torch.float32)


@pytest.mark.parametrize("far", [0, 131071, (1 << 24) + 1, (1 << 31) - 1, -5])
def test_far_positions(cuda_device, far):
    """The angle is reduced exactly: far positions are as close as near ones."""
    batch, qkv, qw, kw = make(cuda_device, [40, 9], [33, 9], 8, 2, 128, 16, seed=5)
    pos = (torch.arange(batch.N) - 40 + far).clamp(-(1 << 31), (1 << 31) - 1).to(torch.int32)
    run(batch, qkv, positions=pos, qw=qw, kw=kw, dtype=torch.float32)


def test_one_row_per_request(cuda_device):
    """q_offsets None: each request's last token; an empty request is skipped without an error."""
    batch, qkv, qw, kw = make(cuda_device, [50, 16, 17, 1], [1, 1, 1, 1], 32, 8, 128, 16, seed=2)
    run(batch, qkv, qw=qw, kw=kw, dtype=torch.float32, offsets=False)
    batch, qkv, qw, kw = make(cuda_device, [50, 0, 17], [1, 0, 1], 8, 2, 64, 16, seed=3, tail=1)
    batch.offs = [0, 1, 1, 2]
    kv = batch.to_device()
    q_out = torch.full((3, 8, 64), 7.0, device=cuda_device)
    B.asp_norm_rotate_append(kv, qkv.to(cuda_device), None, None, qw.to(cuda_device), None, 1e-6,
                             inv_freq_of(64, cuda_device), False, q_out, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    assert bool((q_out[1] == 7.0).all()) and not bool((q_out[[0, 2]] == 7.0).any())


def test_zero_rows_norm_to_zero(cuda_device):
    """A row of zeros has no direction: eps keeps it finite."""
    batch, qkv, qw, kw = make(cuda_device, [20], [20], 8, 2, 64, 16)
    qkv[3:9] = 0
    run(batch, qkv, qw=qw, kw=kw)


def test_many_requests(cuda_device):
    """More requests than a block has threads; ragged, most of them a token or none."""
    tokens = [1 + (i * 7) % 23 for i in range(700)]
    news = [min(t, (i * 5) % 3) for i, t in enumerate(tokens)]
    batch, qkv, qw, kw = make(cuda_device, tokens, news, 4, 2, 64, 16, seed=11)
    run(batch, qkv, qw=qw, kw=kw)


def test_bad_page_and_offsets(cuda_device):
    batch, qkv, qw, kw = make(cuda_device, [40, 20], [40, 20], 8, 2, 64, 16)
    batch.table[0, 1] = batch.n_phys + 5
    kv = batch.to_device()
    k0 = batch.k_dev.clone()
    q_out = torch.zeros((60, 8, 64), dtype=torch.bfloat16, device=cuda_device)
    args = (kv, qkv.to(cuda_device), batch.offs_dev, None, None, None, 1e-6, None, False, q_out,
            batch.ws)
    B.asp_norm_rotate_append(*args)
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_PAGE_RANGE
    assert torch.equal(q_out.cpu(), qkv[:, :8]), "queries are written all the same"
    assert torch.equal(batch.k_dev[int(batch.table[0, 2])].cpu()[:, :8],
                       qkv[32:40, 8:10].transpose(0, 1))
    for offs in ([0, 41, 61], [0, 30, 20], [-1, 40, 60], [0, 40, 62]):
        batch.k_dev.copy_(k0)
        batch.offs_dev.copy_(torch.tensor(offs, dtype=torch.int32))
        B.asp_norm_rotate_append(*args)
        assert B.asp_get_device_error(batch.ws) & B.ASP_DEVERR_OFFSET_RANGE


@pytest.mark.parametrize("tokens,new", [(1, 1), (40, 40), (37, 5), (33, 1)])
def test_summaries_of_nan_keys(cuda_device, tokens, new):
    """NaN in all keys of a page, or in its only one: as a bulk summary of them."""
    batch = R.Batch(cuda_device, [tokens], [new], 8, 2, 64, 16, seed=3)
    kv = batch.to_device()
    old = torch.tensor([tokens - new], dtype=torch.int32, device=cuda_device)
    before = B.PagedKV(batch.k_dev, batch.v_dev, batch.summ_dev, batch.table_dev, old, 8)
    B.asp_page_summarize(before, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    qkv = torch.randn((new, 12, 64), generator=batch.gen).to(torch.bfloat16)
    qkv[:, 8:10, 12:17] = math.nan
    qkv[-1, 9] = math.nan
    q_out = torch.zeros((new, 8, 64), dtype=torch.bfloat16, device=cuda_device)
    B.asp_norm_rotate_append(kv, qkv.to(cuda_device), batch.offs_dev, None, None, None, 1e-6, None,
                             False, q_out, batch.ws)
    got = batch.summ_dev.clone()
    B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    assert torch.equal(torch.isnan(got), torch.isnan(batch.summ_dev))
    assert torch.equal(got.nan_to_num(0.5), batch.summ_dev.nan_to_num(0.5))
