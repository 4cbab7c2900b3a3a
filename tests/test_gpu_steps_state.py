"""DecodeStep and ChunkStep where layers or caches do not fit together, and weights behind a prefix."""

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from adaptive_sparse_paged_gb300.step import ChunkStep, DecodeStep
from tests import prompt_ref as R
from tests import q8_ref as Q

pytestmark = pytest.mark.gpu


def test_staging_goes_with_every_layer(cuda_device):
    """Each layer's tokens are read back by its own lengths and attended over by staging's: a later
    layer with lengths, a batch or pages of its own is refused like the first."""
    dev = cuda_device
    layers = [Q.Q8Batch(dev, [20, 9], [5, 9], 8, 2, 64, 16, seed=s) for s in (1, 2)]
    kvs = [b.to_device() for b in layers]
    other = Q.Q8Batch(dev, [20, 9, 3], [5, 9, 0], 8, 2, 64, 16, seed=3).to_device()
    lens = kvs[0].seq_lens
    same = B.QuantPagedKV(kvs[1].k_cache, kvs[1].v_cache, kvs[1].scales, kvs[1].summaries,
                          kvs[1].block_table, lens, 8)
    k, v = (torch.zeros((8, 2, 16, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
    staging = B.PagedKV(k, v, kvs[0].summaries, table, lens, 8)
    qkv = torch.zeros((2, 14, 12, 64), dtype=torch.bfloat16, device=dev)
    offs = layers[0].offs_dev
    ChunkStep([kvs[0], same], qkv, offs, staging=staging)
    for bad in (kvs[1], other):
        with pytest.raises(ValueError, match="staging"):
            ChunkStep([kvs[0], bad], qkv, offs, staging=staging)
    plain = B.PagedKV(k, v, kvs[0].summaries, table, lens, 8)
    with pytest.raises(ValueError, match="8-bit"):
        ChunkStep([kvs[0], plain], qkv, offs, staging=staging)
    q = torch.zeros((2, 2, 8, 64), device=dev)
    with pytest.raises(ValueError, match="8-bit"):
        DecodeStep([kvs[0], plain], q, 0.9)


@pytest.mark.parametrize("d,gamma", [(64, 0.9), (128, 1.0)])
def test_weights_behind_a_prefix(cuda_device, d, gamma):
    """What every cached token received of attention over the prefix and the own tokens together:
    its probability among both, which the own tokens' lse alone would make too large.

    Bound: a weight is exp(s - lse). s is d products in fp32 of bf16 numbers, the queries in three
    bf16 terms (24 bits); the own lse has them in two (2^-17), the prefix's as they are (bf16
    numbers here); sums of under 300 terms, logarithms and exponentials are a few fp32 steps."""
    dev = cuda_device
    own = [R.Batch(dev, [70, 33, 5], [0] * 3, 8, 2, d, 16, seed=s) for s in (1, 2)]
    pre = [R.Batch(dev, [200, 1], [2, 1], 8, 2, d, 16, seed=s) for s in (3, 4)]
    kvs, pkvs = [b.to_device() for b in own], [b.to_device() for b in pre]
    for b, kv in zip(own, kvs):
        B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, b.ws)
    rows = torch.tensor([0, 2, 3], dtype=torch.int32, device=dev)
    q16 = torch.randn((2, 3, 8, d), generator=own[0].gen).to(torch.bfloat16)
    q32 = q16.float()
    weights = torch.zeros((2,) + tuple(kvs[0].weights_shape), device=dev)
    step = DecodeStep(kvs, q32.to(dev), gamma, weights=weights,
                      prefix=(pkvs, rows, q16.to(dev)))
    step.run()
    assert B.asp_get_device_error(step.ws) == 0 and B.asp_get_device_error(step.prefix_ws) == 0
    lists, counts = step.lists.cpu(), step.lens.cpu()
    for l in range(2):
        for r in range(3):
            group, T = (0, 0, 1)[r], own[l].tokens[r]
            for h in range(2):
                ids = lists[l, r, h, :int(counts[l, r, h])].long()
                at = (ids[:, None] * 16 + torch.arange(16)).flatten()
                at = at[at < T]
                heads = slice(4 * h, 4 * h + 4)
                q = q32[l, r, heads].double()
                k = own[l].rows(own[l].k, r)[at, h].double()
                pk = pre[l].rows(pre[l].k, group)[:, h].double()
                x, px = q @ k.T * step.sm_scale, q @ pk.T * step.sm_scale
                size = torch.cat([(q.abs() @ y.abs().T * step.sm_scale).flatten() for y in (k, pk)]).max()
                lse = torch.logsumexp(torch.cat([x, px], 1), 1)
                want = torch.zeros(T, dtype=torch.float64)
                want[at] = torch.exp(x - lse[:, None]).sum(0)
                dx = (2 * (d + 8) * 2.0 ** -23 + 2.0 ** -17) * size + 2.0 ** -18 + 300 * 2.0 ** -23
                R.close(weights[l, r, h, :T], want, 2 * dx * want + 1e-30, f"weights {l} {r} {h}")
                if group == 0:  # the prefix of one token takes little
                    alone = torch.exp(x - torch.logsumexp(x, 1)[:, None]).sum(0)
                    assert bool((alone > want[at] * (1 + 4 * dx)).all())


@pytest.mark.parametrize("offsets,weights", [([0, 3], True), ([1, 3], True), ([0, 2], False), ([2, 2], True)])
def test_requests_without_a_group(cuda_device, offsets, weights):
    """Requests that row_offsets leaves out have no prefix: what is joined is their own attention,
    rounded once, and their weights go by it."""
    dev = cuda_device
    own = R.Batch(dev, [70, 33, 5], [0] * 3, 8, 2, 64, 16, seed=1)
    pre = R.Batch(dev, [200], [1], 8, 2, 64, 16, seed=3)
    kv, pkv = own.to_device(), pre.to_device()
    B.asp_page_summarize(kv, B.ASP_SUMMARIZE_BULK, None, None, own.ws)
    q16 = torch.randn((1, 3, 8, 64), generator=own.gen).to(torch.bfloat16).to(dev)
    rows = torch.tensor(offsets, dtype=torch.int32, device=dev)
    got = []
    for prefix in ((([pkv]), rows, q16), None):
        w = torch.zeros((1,) + tuple(kv.weights_shape), device=dev) if weights else None
        step = DecodeStep([kv], q16.float(), 0.9, weights=w, prefix=prefix)
        step.capture()
        for _ in range(2):
            if w is not None:
                w.zero_()
            step.replay()
        assert B.asp_get_device_error(step.ws) == 0
        assert prefix is None or B.asp_get_device_error(step.prefix_ws) == 0
        got.append((step, w))
    (step, w), (plain, w0) = got
    for r in range(3):
        joined = offsets[0] <= r < offsets[1]
        same = torch.equal(step.joined[0, r], plain.out[0, r].to(torch.bfloat16))
        assert same != joined and torch.equal(step.joined_lse[0, r], plain.lse[0, r]) != joined
        assert w is None or torch.equal(w[0, r], w0[0, r]) != joined
