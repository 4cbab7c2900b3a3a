"""Workspaces: what each call asks of their size."""

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R

pytestmark = pytest.mark.gpu


def size_without_chunk_calls(kv):
    """The size that a workspace had before the chunk calls' joins and partials came to its end:
    error word, arrivals, scores and the decode's partials, each on a 256-byte boundary."""
    def up(x):
        return -(-x // 256) * 256

    sms = torch.cuda.get_device_properties(kv.device).multi_processor_count
    S = kv.batch * kv.num_kv_heads
    scores = up(256 + 4 * S)
    partials = up(scores + 4 * S * kv.max_pages)
    return up(partials + 4 * (S + sms) * (2 * 8 + 8 * kv.head_dim))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (32, 8, 128)])
def test_only_the_chunk_calls_need_the_end(cuda_device, Hq, Hkv, d):
    dev = cuda_device
    batch = R.Batch(dev, [300, 70], [3, 1], Hq, Hkv, d, 16, seed=3)
    kv = batch.to_device()
    n = size_without_chunk_calls(kv)
    assert n < B.asp_workspace_size(kv)
    small = guards.guarded((n,), torch.uint8, dev, what="workspace without its end")
    short = small[:n - 256]
    B.asp_workspace_init(small)
    B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, batch.ws)
    q = torch.randn((2, Hq, d), generator=batch.gen).to(dev)
    qkv = torch.randn((batch.N, Hq + 2 * Hkv, d), generator=batch.gen).to(torch.bfloat16).to(dev)
    q16 = torch.zeros((batch.N, Hq, d), dtype=torch.bfloat16, device=dev)
    rows_lse = torch.zeros((batch.N, Hq), device=dev)
    new = torch.zeros((2, Hkv, d), dtype=torch.bfloat16, device=dev)
    w = B.new_weights(kv)
    kept = torch.zeros((2, Hkv, 64), dtype=torch.int32, device=dev)
    new_lens = torch.zeros(2, dtype=torch.int32, device=dev)

    def calls(ws):
        lists = torch.zeros(kv.lists_shape, dtype=torch.int32, device=dev)
        lens = torch.zeros(kv.lens_shape, dtype=torch.int32, device=dev)
        scores = torch.zeros(kv.lists_shape, device=dev)
        out, lse = torch.zeros_like(q), torch.zeros((2, Hq), device=dev)
        yield lambda: B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, ws)
        yield lambda: B.asp_page_scores(kv, q, scores, ws)
        yield lambda: B.asp_coverage_select_append(kv, new, new, q, 0.9, 0, lists, lens, ws)
        yield lambda: B.asp_coverage_select(kv, q, 0.9, 0, lists, lens, ws)
        yield lambda: B.asp_sparse_decode(kv, q, lists, lens, batch.scale, out, lse, ws)
        yield lambda: B.asp_decode_weights(kv, q, lists, lens, lse, batch.scale, 1.0, None, w, ws)
        yield lambda: B.asp_norm_rotate_append(kv, qkv, batch.offs_dev, None, None, None, 1e-6, None,
                                               False, q16, ws)
        yield lambda: B.asp_weight_evict(kv, w, 64, 8, batch.table_dev, w, kept, new_lens, ws)

    def chunk_calls(ws):
        out = torch.zeros_like(q16)
        yield lambda: B.asp_chunk_attention(kv, q16, batch.offs_dev, batch.scale, out, rows_lse, ws)
        yield lambda: B.asp_chunk_weights(kv, q16, batch.offs_dev, rows_lse, batch.scale, 1.0, None, w,
                                          ws)

    for call in calls(small):
        call()
    assert B.asp_get_device_error(small) == 0
    for call in chunk_calls(batch.ws):
        call()
    assert B.asp_get_device_error(batch.ws) == 0
    for call in [*calls(short), *chunk_calls(small), *chunk_calls(batch.ws[:-256])]:
        with pytest.raises(B.AspError) as e:
            call()
        assert e.value.status == B.ASP_EWORKSPACE
