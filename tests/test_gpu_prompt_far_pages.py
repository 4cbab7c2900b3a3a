"""The prompt-side and eviction calls on pages beyond 2^31 elements of the cache.

The same tokens in a small cache and at the end of one of 2.3 * 10^9 elements: every result
is the same, bit for bit.
"""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B

pytestmark = pytest.mark.gpu

Hq, Hkv, P, d = 16, 4, 16, 128


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def run(dev, n_phys, first_page):
    gen = torch.Generator(device=dev).manual_seed(3)
    tokens, news, pages = [900, 250], [130, 250], [57, 16]
    max_pages = 57
    table = torch.full((2, max_pages), -1, dtype=torch.int32)
    perm = first_page + torch.randperm(sum(pages) + 41, generator=torch.Generator().manual_seed(4))
    table[0, :57], table[1, :16] = perm[:57], perm[57:73]
    dst = torch.full_like(table, -1)
    dst[0, :25], dst[1, :16] = perm[73:98], perm[98:114]
    k = torch.empty((n_phys, Hkv, P, d), dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    used = torch.cat([table.flatten(), dst.flatten()])
    used = used[used >= 0].long().to(dev)
    k[used] = torch.randn((len(used), Hkv, P, d), generator=gen, device=dev).to(torch.bfloat16)
    v[used] = torch.randn((len(used), Hkv, P, d), generator=gen, device=dev).to(torch.bfloat16)
    summ = torch.zeros((2, Hkv, max_pages, 2, d), dtype=torch.bfloat16, device=dev)
    offs = torch.tensor([0, 130, 380], dtype=torch.int32, device=dev)
    old = torch.tensor([t - n for t, n in zip(tokens, news)], dtype=torch.int32, device=dev)
    lens = torch.tensor(tokens, dtype=torch.int32, device=dev)
    table, dst = table.to(dev), dst.to(dev)
    before = B.PagedKV(k, v, summ, table, old, Hq)
    kv = B.PagedKV(k, v, summ, table, lens, Hq)
    ws = B.new_workspace(kv)
    B.asp_page_summarize(before, B.ASP_SUMMARIZE_BULK, None, None, ws)
    qkv = torch.randn((380, Hq + 2 * Hkv, d), generator=gen, device=dev).to(torch.bfloat16)
    freq = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().to(dev)
    one = torch.ones(d, dtype=torch.bfloat16, device=dev)
    q = torch.empty((380, Hq, d), dtype=torch.bfloat16, device=dev)
    out, lse = torch.empty_like(q), torch.empty((380, Hq), device=dev)
    w, w2, w3 = B.new_weights(kv), B.new_weights(kv), B.new_weights(kv)
    kept = torch.zeros((2, Hkv, 400), dtype=torch.int32, device=dev)
    new_lens = torch.zeros(2, dtype=torch.int32, device=dev)
    c = 1 / math.sqrt(d)
    B.asp_norm_rotate_append(kv, qkv, offs, None, one, one, 1e-6, freq, False, q, ws)
    B.asp_chunk_attention(kv, q, offs, c, out, lse, ws)
    B.asp_chunk_weights(kv, q, offs, lse, c, 1.0, None, w, ws)
    qd = q[[129, 379]].float().contiguous()
    B.asp_decode_weights(kv, qd, None, None, lse[[129, 379]].contiguous(), c, 0.5, w, w2, ws)
    B.asp_weight_evict(kv, w2, 400, 64, dst, w3, kept, new_lens, ws)
    assert B.asp_get_device_error(ws) == 0
    moved = [x[dst[b, :25 if b == 0 else 16].long()] for x in (k, v) for b in (0, 1)]
    return [q, out, lse, w, w2, w3, kept, new_lens, summ] + moved


def test_far_pages_give_the_same(cuda_device):
    free, _ = torch.cuda.mem_get_info()
    if free < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    pages = 280_000  # 2.3e9 elements each of K and V
    assert pages * Hkv * P * d > 1 << 31
    far = run(cuda_device, pages, pages - 200)
    near = run(cuda_device, 200, 0)
    for i, (x, y) in enumerate(zip(far, near)):
        assert torch.equal(bits(x), bits(y)), i
