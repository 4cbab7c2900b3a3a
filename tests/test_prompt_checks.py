"""Host-side refusals of the prompt-side and eviction calls, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from adaptive_sparse_paged_gb300 import binding as B
from tests.test_abi_exports import lib  # noqa: F401  (fixture)
from tests.test_host_checks import FAKE, kv

F = ctypes.c_float


def norm(lib, s, **o):
    a = dict(qkv=FAKE, offs=FAKE, n=5, pos=None, qw=FAKE, kw=FAKE, eps=1e-6, freq=FAKE, rot=64,
             inter=0, q16=FAKE, q32=None, ws=FAKE, size=1 << 20)
    a.update(o)
    return lib.asp_norm_rotate_append(ctypes.byref(s), a["qkv"], a["offs"], a["n"], a["pos"], a["qw"],
                                      a["kw"], F(a["eps"]), a["freq"], a["rot"], a["inter"],
                                      a["q16"], a["q32"], a["ws"], a["size"], None)


def attend(lib, s, **o):
    a = dict(q=FAKE, offs=FAKE, n=5, scale=0.1, out=FAKE, lse=FAKE, ws=FAKE, size=1 << 20)
    a.update(o)
    return lib.asp_chunk_attention(ctypes.byref(s), a["q"], a["offs"], a["n"], F(a["scale"]), a["out"],
                                   a["lse"], a["ws"], a["size"], None)


def chunk(lib, s, **o):
    a = dict(q=FAKE, offs=FAKE, n=5, lse=FAKE, scale=0.1, decay=1.0, w_in=FAKE, w_out=FAKE, ws=FAKE,
             size=1 << 20)
    a.update(o)
    return lib.asp_chunk_weights(ctypes.byref(s), a["q"], a["offs"], a["n"], a["lse"], F(a["scale"]),
                                 F(a["decay"]), a["w_in"], a["w_out"], a["ws"], a["size"], None)


def decode(lib, s, **o):
    a = dict(q=FAKE, lists=FAKE, lens=FAKE, lse=FAKE, scale=0.1, decay=1.0, w_in=FAKE, w_out=FAKE,
             ws=FAKE, size=1 << 20)
    a.update(o)
    return lib.asp_decode_weights(ctypes.byref(s), a["q"], a["lists"], a["lens"], a["lse"],
                                  F(a["scale"]), F(a["decay"]), a["w_in"], a["w_out"], a["ws"],
                                  a["size"], None)


def evict(lib, s, **o):
    a = dict(w=FAKE, keep=10, recent=2, dst=FAKE, w_out=FAKE, kept=FAKE, lens=FAKE + 64, ws=FAKE,
             size=1 << 20)
    a.update(o)
    return lib.asp_weight_evict(ctypes.byref(s), a["w"], a["keep"], a["recent"], a["dst"], a["w_out"],
                                a["kept"], a["lens"], a["ws"], a["size"], None)


CALLS = (norm, attend, chunk, decode, evict)


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("over,want", [
    (dict(k_cache=None), B.ASP_EINVAL), (dict(batch=0), B.ASP_EINVAL),
    (dict(num_q_heads=6, num_kv_heads=4), B.ASP_EINVAL), (dict(head_dim=96), B.ASP_EUNSUPPORTED),
    (dict(page_size=8), B.ASP_EUNSUPPORTED), (dict(k_cache=FAKE + 8), B.ASP_EINVAL)])
def test_bad_caches(lib, call, over, want):
    assert call(lib, kv(**over)) == want


@pytest.mark.parametrize("call", CALLS)
def test_bad_workspaces(lib, call):
    for ws in (None, FAKE + 16):
        assert call(lib, kv(), ws=ws) == B.ASP_EWORKSPACE


@pytest.mark.parametrize("call,over", [
    (norm, dict(qkv=None)), (norm, dict(qkv=FAKE + 2)), (norm, dict(n=-1)),
    (norm, dict(offs=None)),                       # one row a request needs num_tokens == batch
    (norm, dict(q16=None)), (norm, dict(q16=FAKE + 8)), (norm, dict(q32=FAKE + 4)),
    (norm, dict(eps=-1.0)), (norm, dict(eps=float("nan"))), (norm, dict(rot=130)),
    (norm, dict(rot=-8)), (norm, dict(rot=12)), (norm, dict(freq=None)), (norm, dict(inter=2)),
    (norm, dict(qw=FAKE + 2)), (norm, dict(kw=FAKE + 4)),
    (attend, dict(q=None)), (attend, dict(q=FAKE + 8)), (attend, dict(offs=None)),
    (attend, dict(n=-3)), (attend, dict(out=None)), (attend, dict(out=FAKE + 8)),
    (attend, dict(lse=None)), (attend, dict(scale=0.0)), (attend, dict(scale=float("inf"))),
    (attend, dict(scale=float("nan"))),
    (chunk, dict(q=None)), (chunk, dict(offs=None)), (chunk, dict(lse=None)),
    (chunk, dict(w_out=None)), (chunk, dict(decay=-0.5)), (chunk, dict(decay=float("nan"))),
    (chunk, dict(scale=-1.0)), (chunk, dict(w_in=FAKE + 4)), (chunk, dict(w_out=FAKE + 8)),
    (decode, dict(q=None)), (decode, dict(q=FAKE + 4)), (decode, dict(lists=None)),
    (decode, dict(lens=None)), (decode, dict(lse=None)), (decode, dict(w_out=None)),
    (decode, dict(decay=float("inf"))), (decode, dict(scale=0.0)),
    (evict, dict(w=None)), (evict, dict(dst=None)), (evict, dict(w_out=None)),
    (evict, dict(kept=None)), (evict, dict(lens=None)), (evict, dict(lens=FAKE)),  # = seq_lens
    (evict, dict(keep=0)), (evict, dict(keep=64 * 16 + 1)), (evict, dict(recent=-1)),
    (evict, dict(recent=11)), (evict, dict(w=FAKE + 4)), (evict, dict(w_out=FAKE + 4)),
])
def test_bad_arguments(lib, call, over):
    assert call(lib, kv(), **over) == B.ASP_EINVAL


def test_too_many_rows(lib):
    n = B.ASP_MAX_NEW_TOKENS + 1
    for call in (norm, attend, chunk):
        assert call(lib, kv(), n=n) == B.ASP_EUNSUPPORTED


def test_a_scale_that_overflows_the_chunk_weights(lib):
    """lse / sm_scale is formed in fp32: a scale that could make it infinite is refused."""
    for scale in (2.0 ** -101, 1e-38, 1e-45):
        assert chunk(lib, kv(), scale=scale) == B.ASP_EINVAL
    # the smallest one passes this check and meets the next
    assert chunk(lib, kv(), scale=2.0 ** -100, ws=None) == B.ASP_EWORKSPACE
    assert decode(lib, kv(), scale=1e-38, ws=None) == B.ASP_EWORKSPACE
