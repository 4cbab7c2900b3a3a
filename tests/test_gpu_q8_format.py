"""8-bit pages with bytes that no append writes but the format defines: any scale byte below 255."""

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import prompt_ref as R
from tests import q8_ref as Q
from tests import test_gpu_q8_decode as TD

pytestmark = pytest.mark.gpu


def small_rows(batch, row, bytes_):
    """Every token's row of K (0) or V (1): codes of magnitude 1 and up (56 is e4m3's 1), scale
    bytes among `bytes_`. All their values are bf16 numbers."""
    for b, t in enumerate(batch.tokens):
        for s in range(t):
            ph, at = int(batch.table[b, s // batch.P]), s % batch.P
            codes = torch.randint(56, 0x7f, (batch.Hkv, batch.d), generator=batch.gen)
            codes += 128 * torch.randint(0, 2, codes.shape, generator=batch.gen)
            pick = torch.randint(0, len(bytes_), (batch.Hkv,), generator=batch.gen)
            scales = torch.tensor(bytes_, dtype=torch.uint8)[pick]
            (batch.v8 if row else batch.k8)[ph, :, at] = codes.to(torch.uint8)
            batch.scales[ph, :, row, at] = scales
            vals = Q.values(codes.to(torch.uint8), scales)
            (batch.v if row else batch.k)[ph, :, at] = vals.to(torch.bfloat16)
            assert torch.equal((batch.v if row else batch.k)[ph, :, at].double(), vals)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (8, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("bytes_", [[0], [0, 1, 2], [1]])
def test_smallest_scales_of_keys(cuda_device, Hq, Hkv, d, bytes_):
    """A byte of 0 is 2^-127, as in the pages read back: with queries as large as fp32 holds, such
    keys have logits that count."""
    batch = Q.Q8Batch(cuda_device, [40, 17], [0, 0], Hq, Hkv, d, 16, seed=d + Hkv)
    small_rows(batch, 0, bytes_)
    q = torch.randn((2, Hq, d), generator=batch.gen) * 2.0 ** 119 / d ** 0.5
    lists, lens = TD.random_lists(batch, 1.0)
    _, lse = TD.run(batch, lists, lens, q=q, scale=0.5)
    o, _, tol, _ = TD.definition(batch, q, lists, lens, 0.5)
    even, _, _, _ = TD.definition(batch, torch.zeros_like(q), lists, lens, 0.5)
    assert bool(((even - o).abs() > tol).any()), "logits of zero would be within the bound"
    # the same values read back into bf16 pages
    k, v = (torch.zeros((batch.n_phys, Hkv, 16, d), dtype=torch.bfloat16, device=cuda_device)
            for _ in range(2))
    B.asp_q8_read(batch.kv, k, v, batch.table_dev, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    for b, t in enumerate(batch.tokens):
        assert torch.equal(batch.rows(k.cpu(), b), batch.rows(batch.k, b))
