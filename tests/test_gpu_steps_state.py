"""DecodeStep and ChunkStep where layers or caches do not fit together."""

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from adaptive_sparse_paged_gb300.step import ChunkStep, DecodeStep
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
