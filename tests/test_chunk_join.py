"""Joins of items that several thread blocks share: nothing but this call's own is followed.

A workspace keeps what earlier calls left in it, perhaps of another operator or shape. A CTA
whose bounded wait gives up must not leave such a join behind, and the joining kernels follow
none that names something outside the call.
"""

import ctypes
import os
import subprocess

import pytest
import torch

from adaptive_sparse_paged_gb300 import binding as B
from adaptive_sparse_paged_gb300 import build
from tests import prompt_ref as R
from tests.test_gpu_chunk_attention import call

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    try:
        nvcc = build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path_factory.mktemp("probe") / "probe.so"
    cmd = [nvcc, "-shared", *build.compile_flags(), "-cudart", "shared", "-Xlinker",
           "-rpath," + build._cuda_lib_dir(nvcc), os.path.join(HERE, "chunk_join_probe.cu"),
           "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise AssertionError(r.stderr)
    return ctypes.CDLL(str(out))


def test_only_joins_of_the_call_are_followed(probe):
    good = dict(b=3, h=1, item=4, pieces=5, batch=4, kv_heads=2, cta=10, ctas=15)

    def valid(**o):
        return probe.join_valid(*(dict(good, **o)[k] for k in good)) != 0

    assert valid() and valid(item=0) and valid(pieces=2) and valid(cta=0, ctas=5)
    for bad in (dict(b=4), dict(b=-1), dict(b=1 << 30), dict(h=2), dict(h=-1), dict(item=-1),
                dict(pieces=0), dict(pieces=1), dict(pieces=-3), dict(pieces=6), dict(cta=11),
                dict(pieces=1 << 30)):
        assert not valid(**bad), bad


@pytest.mark.gpu
def test_a_wait_that_gives_up_leaves_no_join(cuda_device, probe):
    """Nobody takes the pieces: the handing thread gives up (about 2 s) and a join of an earlier
    call is gone."""
    batch, ctas = 40, 4  # ten pieces a CTA, more than the ring holds
    offs = torch.arange(batch + 1, dtype=torch.int32, device=cuda_device)
    lens = torch.ones(batch, dtype=torch.int32, device=cuda_device)
    joins = torch.tensor([[99, 7, 5, 3]] * (ctas + 1), dtype=torch.int32, device=cuda_device)
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    torch.cuda.synchronize()
    ptr = [ctypes.c_void_p(t.data_ptr()) for t in (offs, lens, joins, err)]
    assert probe.hand_out_to_nobody(ptr[0], ptr[1], batch, 1, batch, ctas, ptr[2], ptr[3]) == 0
    assert int(err) == B.ASP_DEVERR_TIMEOUT
    assert joins.tolist() == [[0, 0, 0, 0]] * ctas + [[99, 7, 5, 3]]


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["attend", "weigh"])
def test_nothing_is_joined_after_a_timeout(cuda_device, op):
    """With the timeout bit set, partials may be an earlier call's: shared rows stay as they were."""
    # every item of the call is shared: one item of 40 units, or three of 18 in all
    tokens, new = (5000, 3) if op == "attend" else (600, 600)
    batch = R.Batch(cuda_device, [tokens], [new], 2, 1, 64, 16, seed=1)
    batch.to_device()
    q, lse = batch.q.to(cuda_device), torch.zeros((batch.N, 2), device=cuda_device)

    def run():
        if op == "attend":
            return call(batch)[0]
        w = torch.full((1, 1, batch.max_pages * 16), 7.0, device=cuda_device)
        B.asp_chunk_weights(batch.kv, q, batch.offs_dev, lse, batch.scale, 1.0, None, w, batch.ws)
        return w[0, 0, :tokens]

    want = run()
    assert B.asp_get_device_error(batch.ws) == 0 and not bool((want == 7.0).any())
    batch.ws.view(torch.int32)[0] = B.ASP_DEVERR_TIMEOUT
    got = run()
    assert B.asp_get_device_error(batch.ws) == B.ASP_DEVERR_TIMEOUT
    assert bool((got == 7.0).all())
    B.asp_workspace_init(batch.ws)
    assert torch.equal(run(), want)
    assert B.asp_get_device_error(batch.ws) == 0
