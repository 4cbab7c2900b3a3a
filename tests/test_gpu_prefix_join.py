"""asp_prefix_attention's join of a row's two parts, where their sizes are extreme."""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R
from tests import q8_ref as Q
from tests import test_gpu_q8_decode as TD

pytestmark = pytest.mark.gpu


def outputs(batch):
    out = guards.guarded((batch.N, batch.Hq, batch.d), torch.bfloat16, batch.dev, fill=7.0, what="out")
    lse = guards.guarded((batch.N, batch.Hq), torch.float32, batch.dev, fill=7.0, what="lse")
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,rows", [([3000], [5]), ([40, 0], [700, 3]), ([2100, 900], [100, 300])])
@pytest.mark.parametrize("q_size", [1.0, 300.0, 30000.0])
def test_no_own_tokens_is_no_own_part(cuda_device, d, tokens, rows, q_size):
    """Rows whose own lse is -inf: bit for bit what the call gives without own parts, however
    large the logits (pieces that are whole items, and that are joined)."""
    batch = R.Batch(cuda_device, tokens, rows, 8, 2, d, 16, seed=d)
    kv = batch.to_device()
    q = (batch.q.float() * q_size).to(torch.bfloat16).to(cuda_device)
    own_out = torch.full((batch.N, 8, d), math.nan, device=cuda_device)
    own_lse = torch.full((batch.N, 8), -math.inf, device=cuda_device)
    got = []
    for own in ((None, None), (own_out, own_lse)):
        out, lse = outputs(batch)
        B.asp_prefix_attention(kv, q, batch.offs_dev, batch.scale, *own, out, lse, batch.ws)
        got.append((out, lse))
    assert B.asp_get_device_error(batch.ws) == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 40, 5000])
@pytest.mark.parametrize("base", [0.0, 40000.0, 1e6, -1e6])
def test_weights_sum_to_one(cuda_device, d, T, base):
    """Both parts are one bf16 vector, so that the result is: however large the logits, from whose
    rounded lse the weights would be off by 2^-24 of it each.

    All keys are equal and a logit times log2(e) is a whole number that fp32 holds, so that every
    probability is 1, the prefix's sum T and its O T times the vector, all exactly. The rest, two
    exponentials, their sum, two divisions and one multiply-add, is under 2^-20 of the vector:
    less than half a step of bf16."""
    batch = R.Batch(cuda_device, [T], [4], 8, 2, d, 16, seed=T)
    value = torch.linspace(-3, 3, d).to(torch.bfloat16)
    key = torch.zeros((T, 2, d), dtype=torch.bfloat16)
    key[..., 0] = 1.0
    batch.put(batch.k, 0, key)
    batch.put(batch.v, 0, value.expand(T, 2, d))
    kv = batch.to_device()
    q = torch.zeros((4, 8, d), dtype=torch.bfloat16)
    q[..., 0] = 8 * base
    scale = float(torch.tensor(math.log(2.0), dtype=torch.float32)) / 8
    pre = float(q[0, 0, 0]) * scale + math.log(T)
    own_lse = (pre + torch.tensor([1.0, -1.0, 0.0, 3.0])[:, None]).expand(4, 8).float().contiguous()
    own_out = value.float().expand(4, 8, d).contiguous()
    out, lse = outputs(batch)
    B.asp_prefix_attention(kv, q.to(cuda_device), batch.offs_dev, scale, own_out.to(cuda_device),
                           own_lse.to(cuda_device), out, lse, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    assert torch.equal(out.cpu(), value.expand(4, 8, d))
    both = torch.logaddexp(torch.full((4, 8), pre, dtype=torch.float64), own_lse.double())
    R.close(lse, both, 4 * R.FP32 * both.abs() + 2.0 ** -18, "lse")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens,rows", [([3000], [5]), ([40], [700])])
def test_nan_of_an_own_part_shows(cuda_device, d, tokens, rows):
    """A NaN in own_out counts wherever its row has own tokens, be their weight too small for fp32:
    in items that are joined and in whole ones alike. Where own_lse is -inf it does not."""
    batch = R.Batch(cuda_device, tokens, rows, 8, 2, d, 16, seed=d)
    kv = batch.to_device()
    own_out = torch.zeros((batch.N, 8, d), device=cuda_device)
    own_out[..., 7] = math.nan
    own_lse = torch.full((batch.N, 8), -300.0, device=cuda_device)
    own_lse[1::2] = -math.inf
    for half in (False, True):
        out, lse = outputs(batch)
        part = own_out.to(torch.bfloat16) if half else own_out
        B.asp_prefix_attention(kv, batch.q.to(cuda_device), batch.offs_dev, batch.scale, part, own_lse,
                               out, lse, batch.ws)
        assert B.asp_get_device_error(batch.ws) == 0
        nan = torch.zeros((batch.N, 8, d), dtype=torch.bool)
        nan[0::2, :, 7] = True
        assert torch.equal(out.isnan().cpu(), nan) and bool(lse.isfinite().all())


def test_one_workspace_for_the_own_caches_too(cuda_device):
    """The prefix call in the workspace of the decode whose results it joins, of another shape:
    both give what they give in workspaces of their own, call after call."""
    own = Q.Q8Batch(cuda_device, [4000] + [60] * 90, [0] * 91, 8, 2, 64, 16, seed=2)
    batch = R.Batch(cuda_device, [2500, 40], [90, 1], 8, 2, 64, 16, seed=3)
    kv, pkv = own.to_device(), batch.to_device()
    lists, lens = (x.to(cuda_device) for x in TD.random_lists(own, 1.0))
    q = batch.q.to(cuda_device)
    shared = guards.guarded((max(own.ws.numel(), batch.ws.numel()),), torch.uint8, cuda_device,
                            what="one workspace")
    B.asp_workspace_init(shared)
    results = []
    for ws, pws in ((own.ws, batch.ws), (shared, shared)):
        for _ in range(3):
            o, ol = torch.zeros((91, 8, 64), device=cuda_device), torch.zeros((91, 8), device=cuda_device)
            out, lse = outputs(batch)
            B.asp_q8_decode(kv, q.float(), lists, lens, 0.125, o, ol, ws)
            B.asp_prefix_attention(pkv, q, batch.offs_dev, 0.125, o, ol, out, lse, pws)
            assert B.asp_get_device_error(ws) == 0 and B.asp_get_device_error(pws) == 0
            results.append([x.clone() for x in (o, ol, out, lse)])
    for r in results[1:]:
        for x, y in zip(r, results[0]):
            assert torch.equal(x, y)


def test_no_rows_with_own_parts(cuda_device):
    """A call without rows, own parts or not, is fine; buffers that overlap are refused."""
    batch = R.Batch(cuda_device, [20, 7], [3, 1], 8, 2, 64, 16, seed=1)
    kv = batch.to_device()
    none = torch.zeros(3, dtype=torch.int32, device=cuda_device)
    rows, lse = torch.zeros((0, 8, 64), device=cuda_device), torch.zeros((0, 8), device=cuda_device)
    half = rows.to(torch.bfloat16)
    for own in (rows, half):
        B.asp_prefix_attention(kv, half, none, 0.1, own, lse, half.clone(), lse.clone(), batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    q, own_lse = batch.q.to(cuda_device), torch.zeros((4, 8), device=cuda_device)
    both = torch.zeros((4, 8, 64), device=cuda_device)
    inside = both.view(torch.bfloat16).view(-1)[:2048].view(4, 8, 64)
    for out, lse in ((inside, torch.zeros_like(own_lse)), (q, torch.zeros_like(own_lse)),
                     (torch.zeros_like(q), own_lse)):
        with pytest.raises(B.AspError) as e:
            B.asp_prefix_attention(kv, q, batch.offs_dev, 0.1, both, own_lse, out, lse, batch.ws)
        assert e.value.status == B.ASP_EINVAL
