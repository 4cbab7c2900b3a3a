"""Host functions behind the launches, looked at without a GPU."""

import ctypes
import os
import subprocess

import pytest

from adaptive_sparse_paged_gb300 import build
from tests.test_host_checks import kv

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    try:
        nvcc = build._nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    out = tmp_path_factory.mktemp("probe") / "probe.so"
    cmd = [nvcc, "-shared", *build.compile_flags(), "-cudart", "shared", "-Xlinker",
           "-rpath," + build._cuda_lib_dir(nvcc), os.path.join(HERE, "host_probe.cu"), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        raise AssertionError(r.stderr)
    return ctypes.CDLL(str(out))


@pytest.mark.parametrize("over,pages", [({}, True), (dict(k_cache=None, v_cache=None), False)])
def test_selection_prefetches_only_pages_that_are_there(probe, over, pages):
    """The selection fetches the K and V of kept pages ahead of the decode: counted from the
    caches' addresses, so of a cache without bf16 pages it fetches none."""
    there = ctypes.c_int(-1), ctypes.c_int(-1)
    n = probe.select_prefetch(ctypes.byref(kv(**over)), *(ctypes.byref(x) for x in there))
    assert [x.value for x in there] == [int(pages)] * 2
    assert (n > 0) == pages


def test_chunk_parts_lie_behind_all_arrival_counts(probe):
    """The chunk calls' and the prefix call's parts, of whatever shape, never lie where a decode of
    another shape keeps its arrival counts between calls: one workspace can serve both."""
    def parts(**shape):
        at = (ctypes.c_longlong * 4)()
        probe.workspace_parts(ctypes.byref(kv(**shape)), 152, at)
        return list(at)

    shapes = [dict(batch=b, num_kv_heads=h, num_q_heads=h, head_dim=d, max_pages=n)
              for b in (1, 3, 64, 512) for h in (1, 8) for d in (64, 128) for n in (1, 17, 8192)]
    got = [parts(**s) for s in shapes]
    last = max(end for _, end, _, _ in got)
    assert last == 256 + 4 * 4096  # the most segments a call may have
    for begin, end, joins, total in got:
        assert begin == 256 and last <= joins < total
