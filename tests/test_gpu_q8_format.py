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


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (8, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("bytes_", [[0], [0, 3, 9], [240, 244]])
def test_smallest_and_largest_scales_of_values(cuda_device, Hq, Hkv, d, bytes_):
    """Outputs keep their precision where a power of two of theirs is below fp32's normal numbers,
    or its square above the largest."""
    batch = Q.Q8Batch(cuda_device, [40, 17], [0, 0], Hq, Hkv, d, 16, seed=d + Hkv)
    small_rows(batch, 1, bytes_)
    TD.run(batch, *TD.random_lists(batch, 1.0))


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (8, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("T", [1, 17, 700])
@pytest.mark.parametrize("size", [1.0, 1e3, 1e5, 1e9])
def test_one_token_with_all_the_weight(cuda_device, Hq, Hkv, d, T, size):
    """Its value row comes out as it is, however large its logit: the others are 60 and more below
    it, 2^-86 of its weight. Bound: the exponentials of two numbers that cancel, the sums and the
    division, a few fp32 steps; the others' weights, and what the fp16 terms leave of them."""
    batch = Q.Q8Batch(cuda_device, [T], [0], Hq, Hkv, d, 16, seed=T)
    heavy = T // 3
    key = torch.zeros((T, Hkv, d), dtype=torch.float64)
    key[heavy, :, 0] = 1.0
    batch.put8(0, 0, key)
    q = torch.zeros((1, Hq, d))
    q[..., 0] = 60.0 * size / batch.scale
    lists, lens = TD.random_lists(batch, 1.0)
    out, lse = TD.run(batch, lists, lens, q=q)
    want = batch.rows(batch.v, 0)[heavy].double().repeat_interleave(Hq // Hkv, 0)
    rest = T * 2.0 ** -31 * batch.rows(batch.v, 0).double().abs().amax()
    R.close(out[0], want, 2.0 ** -20 * want.abs() + (0 if T == 1 else rest), "out")
    R.close(lse[0], 60.0 * size * torch.ones(Hq, dtype=torch.float64),
            torch.full((Hq,), 2.0 ** -20 * 60 * size, dtype=torch.float64), "lse")


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128), (8, 1, 128), (8, 1, 64)])
@pytest.mark.parametrize("above", [0, 10, 20, 30])
def test_channels_without_the_heavy_row(cuda_device, Hq, Hkv, d, above):
    """One row has a single channel, 2^above larger than all others' values: the other channels are
    held to their own mass and to the stated 2^-32 of the largest weight for each token. (The
    bound by whole rows that other tests use would let the heavy channel excuse them.)"""
    batch = Q.Q8Batch(cuda_device, [90, 33], [0, 0], Hq, Hkv, d, 16, seed=above, spread=0)
    for b, at in ((0, 41), (1, 7)):
        row = torch.zeros((1, Hkv, d), dtype=torch.float64)
        row[..., 3] = 3.0 * 2.0 ** above
        batch.put8(b, 1, row, start=at)
    q = torch.randn((2, Hq, d), generator=batch.gen)
    lists, lens = TD.random_lists(batch, 1.0)
    out, _ = TD.run(batch, lists, lens, q=q)
    o, _, _, _ = TD.definition(batch, q, lists, lens, batch.scale)
    step = 2.0 ** -23
    for b, n in enumerate(batch.tokens):
        k, v = (batch.rows(x, b).double() for x in (batch.k, batch.v))
        slots = torch.arange(n)
        ph = batch.table[b, slots // batch.P].long()
        power = torch.exp2(batch.scales[ph, :, 1, slots % batch.P].double() - 127)
        codes = (v / power[..., None]).abs()
        for head in range(Hq):
            h = head // batch.g
            x = k[:, h] @ q[b, head].double() * batch.scale
            size = (k[:, h].abs() @ q[b, head].double().abs() * batch.scale).max()
            p = torch.softmax(x, 0)
            dx = ((d + 8) * step + 2.0 ** -22) * size + 2.0 ** -20 + n * step
            tol = (2 * dx + n * step) * (p @ v[:, h].abs()) + \
                2.0 ** -32 * (p * power[:, h]).max() * codes[:, h].sum(0)
            R.close(out[b, head], o[b, head], tol, f"out {b} {head}")
