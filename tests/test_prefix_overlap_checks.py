"""asp_prefix_attention refuses buffers that its thread blocks would overwrite under one another."""

import pytest

from adaptive_sparse_paged_gb300 import binding as B
from tests.test_abi_exports import lib  # noqa: F401  (fixture)
from tests.test_host_checks import FAKE, kv
from tests.test_q8_prefix_checks import prefix

S = kv()
N = 5
BF16, FP32, LSE = (N * S.num_q_heads * S.head_dim * 2, N * S.num_q_heads * S.head_dim * 4,
                   N * S.num_q_heads * 4)
STEP = 1 << 20  # buffers that far apart do not touch
APART = dict(q=FAKE, own=FAKE + STEP, own_lse=FAKE + 2 * STEP, out=FAKE + 3 * STEP, lse=FAKE + 4 * STEP,
             n=N, ws=FAKE, size=1 << 20)


@pytest.mark.parametrize("over,good", [
    ({}, True),
    (dict(out=APART["q"]), False),                                  # out in q's place
    (dict(out=APART["q"] + BF16 - 16), False),                      # their ends meet
    (dict(out=APART["q"] + BF16), True),
    (dict(q=APART["out"] + BF16 - 16), False),
    (dict(out=APART["own"]), False),                                # bf16 rows over fp32 ones
    (dict(out=APART["own"] + FP32 - 16), False),
    (dict(out=APART["own"] + FP32), True),
    (dict(out=APART["own"], half=1), True),                         # a bf16 own part's own place
    (dict(out=APART["own"] + 16, half=1), False),
    (dict(out=APART["own"] + BF16, half=1), True),
    (dict(lse=APART["own_lse"]), False),
    (dict(lse=APART["own_lse"] + LSE - 4), False),
    (dict(lse=APART["own_lse"] + LSE), True),
    (dict(own=None, own_lse=None, out=APART["own"]), True),
])
def test_overlaps(lib, over, good):  # noqa: F811
    """What is right comes as far as the workspace, which is too small (on a machine without a GPU:
    as far as the device, which is not there)."""
    got = prefix(lib, S, **{**APART, **over})
    assert (got != B.ASP_EINVAL) == good, got


def test_no_rows_have_no_place(lib):  # noqa: F811
    """A call without rows may give the same address for every buffer: nothing is in them."""
    same = dict(q=FAKE, own=FAKE, own_lse=FAKE, out=FAKE, lse=FAKE, n=0, ws=FAKE, size=1 << 20)
    assert prefix(lib, S, **same) != B.ASP_EINVAL
    assert prefix(lib, S, **{**same, "half": 1}) != B.ASP_EINVAL
