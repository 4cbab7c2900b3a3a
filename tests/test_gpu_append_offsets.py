"""The calls that append, with offsets that do not ascend: what a request gets is all or nothing.

Requests are found by their offsets. Those before the first offset that descends are written
whole, as if the others had no rows; the request where it descends and all behind it are skipped
whole, and the error word says so.
"""

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R
from tests import q8_ref as Q

pytestmark = pytest.mark.gpu

MANY = [3 * b for b in range(41)] + [90] + [123 + 3 * b for b in range(29)]


@pytest.mark.parametrize("call", ["plain", "axes", "q8"])
@pytest.mark.parametrize("Hq,Hkv,d,P", [(8, 2, 64, 16), (32, 8, 128, 64)])
@pytest.mark.parametrize("N,offs,clean", [
    (50, [100, 0, 50], [0, 0, 0]),                    # the first request is wrong
    (50, [0, 50, 10], [0, 50, 50]),                   # the last
    (400, [0, 400, 0, 10], [0, 400, 400, 400]),       # rows that a later request names again
    (400, [7, 300, 290, 400, 350], [7, 300, 300, 300, 300]),
    (50, [0, 30, 60], [0, 30, 30]),                   # past the rows, ascending
    (50, [-4, 20, 50], [20, 20, 50]),                 # before them
    (207, MANY, MANY[:41] + [120] * 30),              # beyond the first 32 requests
])
def test_whole_or_not_at_all(cuda_device, call, Hq, Hkv, d, P, N, offs, clean):
    dev, n_req = cuda_device, len(offs) - 1
    tokens = [17 + max(0, min(N, b) - max(0, a)) for a, b in zip(offs, offs[1:])]
    cls = Q.Q8Batch if call == "q8" else R.Batch
    batch = cls(dev, tokens, [0] * n_req, Hq, Hkv, d, P, seed=n_req)
    qkv = torch.randn((N, Hq + 2 * Hkv, d), generator=batch.gen).to(torch.bfloat16).to(dev)
    freq = (10000.0 ** (-torch.arange(0, d, 2) / d)).float().to(dev)
    axis = (torch.arange(d // 2) % 2).to(torch.int32).to(dev)
    pos = torch.randint(0, 5000, (2, N), generator=batch.gen, dtype=torch.int32).to(dev)
    got = []
    for table in (offs, clean):
        kv = batch.to_device()
        q_out = guards.guarded((N, Hq, d), torch.float32, dev, fill=7.0, what="q_out")
        o = torch.tensor(table, dtype=torch.int32, device=dev)
        norms = (None, None, 1e-6, freq, False, q_out, batch.ws)
        if call == "plain":
            B.asp_norm_rotate_append(kv, qkv, o, pos[0].contiguous(), *norms)
        else:
            append = B.asp_q8_append if call == "q8" else B.asp_norm_rotate_axes_append
            append(kv, qkv, o, pos, axis, *norms)
        err = B.asp_get_device_error(batch.ws)
        assert err == (B.ASP_DEVERR_OFFSET_RANGE if table is offs else 0)
        rest = [batch.scales_dev] if call == "q8" else []
        got.append([x.view(torch.uint8) for x in
                    [q_out, batch.k_dev, batch.v_dev, batch.summ_dev] + rest])
    for name, x, y in zip(("q_out", "k", "v", "summaries", "scales"), *got):
        assert torch.equal(x, y), name
