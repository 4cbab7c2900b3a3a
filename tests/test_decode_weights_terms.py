"""asp_decode_weights takes its fp32 queries in whole: three bf16 terms, not two.

Every key has one channel that is not zero, so that a logit is one product and its error comes
from the query's split and a handful of fp32 roundings. The bound counts those; what a query of
two terms leaves out is up to 2^-18 of the logit and has to break it.
"""

import math

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from tests import guards
from tests import prompt_ref as R

LSE = 45.0


def case(dev, T, g, d, P, seed):
    """Logits of 32 to 50; q of one sign a channel, so that no head's logit is far from LSE."""
    batch = R.Batch(dev, [T], [1], g, 1, d, P, seed=seed)
    sign = torch.randint(0, 2, (d,), generator=batch.gen) * 2.0 - 1.0
    q = (1 + 0.25 * torch.rand((1, g, d), generator=batch.gen)) * sign
    k = torch.zeros((T, 1, d), dtype=torch.bfloat16)
    t = torch.arange(T)
    k[t, 0, t % d] = (40 / batch.scale / 1.125 * sign[t % d]).to(torch.bfloat16)
    batch.put(batch.k, 0, k)
    return batch, q


def weights(batch, q):
    """(weights, bound) [T] in float64 with lse = LSE for every head."""
    k = batch.rows(batch.k, 0)[:, 0].double()
    x = torch.einsum("gd,td->gt", q[0].double(), k) * batch.scale
    p = torch.exp(x - LSE)
    # A logit's error: the split's remainder 2^-27, two additions of the terms' products (exact
    # themselves), the scale's, the constant's and their product's rounding; for the lse, the
    # constant's and the product's; one more for what the exponential is taken of, which is
    # off by two steps itself.
    dx = (2.0 ** -27 + 5 * R.FP32) * x.abs() + 2 * R.FP32 * LSE + R.FP32 * (x - LSE).abs() + 2.0 ** -22
    w = p.sum(0)
    return w, (p * dx).sum(0) * (1 + 2.0 ** -10) + 8 * R.FP32 * w


def in_terms(q, n):
    """The sum of a query's first n bf16 terms, in float64."""
    total, rest = torch.zeros_like(q, dtype=torch.float64), q.clone()
    for _ in range(n):
        term = rest.to(torch.bfloat16).float()
        total, rest = total + term.double(), rest - term
    return total


CASES = [(1500, 1, 128, 16), (700, 1, 64, 32), (900, 4, 128, 64), (1111, 8, 64, 16)]


@pytest.mark.parametrize("T,g,d,P", CASES)
def test_two_terms_would_be_seen(T, g, d, P):
    batch, q = case(torch.device("cpu"), T, g, d, P, seed=T)
    want, tol = weights(batch, q)
    off = [(weights(batch, in_terms(q, n))[0] - want).abs() / tol for n in (2, 3)]
    assert float(off[0].max()) > 2, "a query of two terms passes"
    assert float(off[1].max()) < 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("T,g,d,P", CASES)
def test_queries_enter_in_whole(cuda_device, T, g, d, P, listed):
    batch, q = case(cuda_device, T, g, d, P, seed=T)
    want, tol = weights(batch, q)
    kv = batch.to_device()
    lists = lens = None
    if listed:
        lists = torch.arange(batch.max_pages, dtype=torch.int32, device=cuda_device)[None, None]
        lists = lists.contiguous()
        lens = torch.full((1, 1), batch.max_pages, dtype=torch.int32, device=cuda_device)
    lse = torch.full((1, g), LSE, device=cuda_device)
    w = guards.guarded((1, 1, batch.max_pages * P), torch.float32, cuda_device, fill=5.0)
    B.asp_decode_weights(kv, q.to(cuda_device), lists, lens, lse, batch.scale, 1.0, None, w, batch.ws)
    assert B.asp_get_device_error(batch.ws) == 0
    R.close(w[0, 0, :T].cpu(), want, tol, "weights")
